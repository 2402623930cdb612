"""Cases of the few-token MoE layer (``moe_decode``) and of the linear layer with a
fused epilogue (``moe_linear``): inputs, one pass through each, its work and its
64-bit value.

``own`` False computes the operators in plain torch operations; True makes the
calls of ``sigmoid_top_routing_b200.api``.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- cases -------------------------------------------------------------------
def _moe(name, T, H, E, k, I, fmt="bf16", act="swiglu", Is=0, residual=True, score="sigmoid", norm=True,
         limit=0.0, out_scale=1.0):
    c = {"op": "moe", "T": T, "H": H, "E": E, "k": k, "I": I, "fmt": fmt, "act": act, "Is": Is,
         "residual": residual, "score": score, "norm": norm, "limit": limit, "out_scale": out_scale}
    if name:
        c["name"] = name
    return c


def _lin(name, M, N, K, act="none", bias=False, residual="none", out="bf16"):
    c = {"op": "linear", "M": M, "N": N, "K": K, "act": act, "bias": bias, "residual": residual, "out": out}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the smallest call: one token through a small block, all latency
        _moe("moe_tiny_t1", 1, 256, 8, 2, 128),
        # one sequence decoding through 4-bit experts
        _moe("moe_affine4_t1", 1, 2048, 64, 4, 1536, fmt="affine4"),
        # a few sequences, NVFP4 experts with the input clamp
        _moe("moe_nvfp4_t5", 5, 2048, 64, 4, 1536, fmt="nvfp4", limit=7.0),
        # one sequence, relu^2 experts beside a shared expert, scaled routed sum
        _moe("moe_relu2_shared_t1", 1, 2048, 64, 6, 1024, act="relu2", Is=2048, out_scale=2.5),
        # eight sequences through bf16 experts
        _moe("moe_bf16_t8", 8, 2048, 32, 4, 1792),
        # the most tokens of the range, softmax router without normalisation
        _moe("moe_bf16_t16", 16, 2048, 32, 4, 1792, score="softmax", norm=False, residual=False),
        # one token's output projection with the residual stream
        _lin("linear_m1", 1, 2048, 2048, residual="bf16"),
        # a few tokens' gated up projection with a bias
        _lin("linear_swiglu_m8", 8, 7168, 2048, act="swiglu", bias=True),
        # ragged everything: odd rows, odd features, an inner size off the tile, fp32 residual and output
        _lin("linear_odd_m77", 77, 1537, 1795, bias=True, residual="f32", out="f32"),
        # a chunk of prompt through a relu^2 up projection
        _lin("linear_relu2_m512", 512, 4096, 2048, act="relu2"),
        # a prompt's gated up projection: the largest product
        _lin("linear_swiglu_m8192", 8192, 7168, 2048, act="swiglu"),
        # the matching down projection into the residual stream
        _lin("linear_down_m8192", 8192, 2048, 7168, bias=True, residual="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        T = rng.randint(1, 16)
        H = 64 * _log(rng, 1, min(64, 65536 // T // 64))
        E = _log(rng, 2, 128)
        I = 64 * _log(rng, 1, 40)
        act = rng.choice(["swiglu", "relu2"])
        while E * H * I > 32 * 2048 * 1792:        # no more weights than the largest listed case
            E = max(2, E // 2)
        return _moe(None, T, H, E, rng.randint(1, min(E, 10)), I, fmt=rng.choice(["bf16", "affine4", "nvfp4"]),
                    act=act, Is=rng.choice([0, 0, 64 * _log(rng, 1, 32)]), residual=rng.random() < 0.6,
                    score=rng.choice(["sigmoid", "sigmoid", "softmax"]), norm=rng.random() < 0.8,
                    limit=rng.choice([0.0, 2.0]) if act == "swiglu" else 0.0, out_scale=rng.choice([1.0, 2.5]))
    M, N, K = _log(rng, 1, 8192), _log(rng, 1, 8192), _log(rng, 8, 8192)
    act = rng.choice(["none", "none", "relu2", "swiglu"])
    while M * N * K > 8192 * 7168 * 2048:
        N = max(1, N // 2)
    return _lin(None, M, N, K, act=act, bias=rng.random() < 0.5, residual=rng.choice(["none", "bf16", "f32"]),
                out=rng.choice(["bf16", "bf16", "f32"]))


# ---- inputs ------------------------------------------------------------------
def _affine4(w):
    """fp32 (N, K) -> codes (N, K/8) int32, scale and bias (N, K/64) bf16 (group min/max)."""
    N, K = w.shape
    g = w.view(N, K // 64, 64)
    lo, hi = g.amin(-1), g.amax(-1)
    s, b = ((hi - lo) / 15).bfloat16(), lo.bfloat16()
    q = torch.round((g - b.float()[..., None]) / s.float()[..., None].clamp_min(1e-30)).clamp_(0, 15)
    q = q.view(N, K // 8, 8).to(torch.int32)
    word = q[..., 0].clone()
    for i in range(1, 8):
        word |= q[..., i] << (4 * i)
    return word, s, b


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nvfp4(w):
    """fp32 (N, K) -> codes (N, K/2) uint8, block scales (N, K/16) e4m3 bytes, global scale ()."""
    N, K = w.shape
    g = w.abs().amax() / (6.0 * 448.0)
    b = w.view(N, K // 16, 16)
    s = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    v = b / (s.float() * g).clamp_min(1e-30)[..., None]
    grid = torch.tensor(_E2M1, device=w.device)
    code = torch.bucketize(v.abs(), (grid[1:] + grid[:-1]) / 2)
    code = (code | ((v < 0) & (code > 0)).long() << 3).view(N, K).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.view(torch.uint8), g


def _experts(gen, E, N, K, fmt):
    """Weights ~ N(0, 0.02) of E experts in the format's tensors."""
    if fmt == "bf16":
        out = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
        for e in range(E):
            out[e] = torch.randn((N, K), generator=gen, device=DEV) * 0.02
        return {"w": out}
    parts = [(_affine4 if fmt == "affine4" else _nvfp4)(torch.randn((N, K), generator=gen, device=DEV) * 0.02)
             for _ in range(E)]
    names = ("w", "scale", "bias") if fmt == "affine4" else ("w", "scale", "glob")
    return {n: torch.stack([p[i] for p in parts]) for i, n in enumerate(names)}


def _weights_of(W1, W2, c):
    from sigmoid_top_routing_b200 import abi, api
    return api.ExpertWeights(
        act=abi.MOE_ACT_SWIGLU if c["act"] == "swiglu" else abi.MOE_ACT_RELU2,
        fmt={"bf16": abi.MOE_W_BF16, "affine4": abi.MOE_W_AFFINE4_G64, "nvfp4": abi.MOE_W_NVFP4}[c["fmt"]],
        w1=W1["w"], w2=W2["w"], w1_scale=W1.get("scale"), w2_scale=W2.get("scale"), w1_bias=W1.get("bias"),
        w2_bias=W2.get("bias"), w1_global=W1.get("glob"), w2_global=W2.get("glob"), swiglu_limit=c["limit"])


def _inputs(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        ld = (K + 7) // 8 * 8                       # rows of a user's buffers start on 16 bytes
        rows = 2 * N if c["act"] == "swiglu" else N
        s = {"x": randn(M, ld).bfloat16()[:, :K], "w": (randn(rows, ld) * (1.0 / math.sqrt(K))).bfloat16()[:, :K],
             "bias": randn(rows) * 0.1 if c["bias"] else None, "residual": None}
        if c["residual"] != "none":
            s["residual"] = randn(M, N).to(torch.bfloat16 if c["residual"] == "bf16" else torch.float32)
        return s
    T, H, E, I = c["T"], c["H"], c["E"], c["I"]
    g = 2 if c["act"] == "swiglu" else 1
    s = {"x": randn(T, H).bfloat16(), "wr": randn(E, H) * 0.02,
         "eb": torch.rand(E, generator=gen, device=DEV) * 0.2 - 0.1,
         "residual": randn(T, H).bfloat16() if c["residual"] else None,
         "W1": _experts(gen, E, g * I, H, c["fmt"]), "W2": _experts(gen, E, H, I, c["fmt"]), "S1": None, "S2": None}
    if c["Is"]:
        s["S1"] = _experts(gen, 1, g * c["Is"], H, c["fmt"])
        s["S2"] = _experts(gen, 1, H, c["Is"], c["fmt"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from sigmoid_top_routing_b200 import api
        if case["op"] == "moe":
            s["layer"] = api.DecodeLayer(
                _weights_of(s["W1"], s["W2"], case), s["wr"], s["eb"], E=case["E"], k=case["k"], I=case["I"],
                Ws=_weights_of(s["S1"], s["S2"], case) if case["Is"] else None, Is=case["Is"],
                out_scale=case["out_scale"], score=case["score"], norm_topk=case["norm"], max_tokens=case["T"])
        else:
            s["linear"] = api.moe_linear
            s["out"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    return s


# ---- the plain form ----------------------------------------------------------
def _dequant(W, fmt, pick):
    """fp32 weights (n, N, K) of the experts `pick`."""
    w = W["w"][pick]
    if fmt == "bf16":
        return w.float()
    if fmt == "affine4":
        q = torch.stack([(w >> (4 * i)) & 15 for i in range(8)], -1).float()
        n, N, _, _ = q.shape
        q = q.view(n, N, -1, 64)
        q = q * W["scale"][pick].float()[..., None] + W["bias"][pick].float()[..., None]
        return q.view(n, N, -1)
    q = torch.stack([w & 15, w >> 4], -1).long()
    n, N, _, _ = q.shape
    v = torch.tensor(_E2M1 + [-a for a in _E2M1], device=w.device)[q].view(n, N, -1, 16)
    v = v * W["scale"][pick].view(torch.float8_e4m3fn).float()[..., None]
    return v.view(n, N, -1) * W["glob"][pick][:, None, None]


def _activate(v, act, limit):
    if act == "relu2":
        return torch.clamp_min(v, 0) ** 2
    if act == "none":
        return v
    g, u = v.chunk(2, -1)
    if limit > 0:
        g, u = torch.clamp_max(g, limit), torch.clamp(u, -limit, limit)
    return g / (1 + torch.exp(-g)) * u


def _plain_linear(s, c):
    v = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _activate(v, c["act"], 0.0)
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return {"y": v.to(torch.bfloat16 if c["out"] == "bf16" else torch.float32)}


def _plain_moe(s, c):
    x = s["x"].float()
    L = s["x"].double() @ s["wr"].double().t()          # 64 bits: the picks lie next to borders
    if c["score"] == "sigmoid":
        sc = 1 / (1 + torch.exp(-L))
    else:
        p = torch.exp(L - L.amax(-1, keepdim=True))
        sc = p / p.sum(-1, keepdim=True)
    idx = torch.sort(sc + s["eb"].double(), dim=-1, descending=True, stable=True)[1][:, :c["k"]]
    w = sc.gather(1, idx)
    if c["norm"]:
        w = w / (w.sum(-1, keepdim=True) + 1e-6)
    w = w.float()
    y = torch.zeros_like(x)
    for j in range(c["k"]):                              # one pick of every token at a time
        h = torch.bmm(_dequant(s["W1"], c["fmt"], idx[:, j]), x[:, :, None])[:, :, 0]
        h = _activate(h, c["act"], c["limit"])
        y += w[:, j:j + 1] * torch.bmm(_dequant(s["W2"], c["fmt"], idx[:, j]), h[:, :, None])[:, :, 0]
    y = y * c["out_scale"]
    if c["Is"]:
        first = torch.zeros(1, dtype=torch.long, device=x.device)
        h = _activate(x @ _dequant(s["S1"], c["fmt"], first)[0].t(), c["act"], c["limit"])
        y = y + h @ _dequant(s["S2"], c["fmt"], first)[0].t()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.bfloat16(), "idx": idx.int(), "w": w}


def run(state):
    c = state["case"]
    if own:
        if c["op"] == "moe":
            y, idx, w = state["layer"](state["x"], residual=state["residual"])
            return {"y": y, "idx": idx, "w": w}
        return {"y": state["linear"](state["x"], state["w"], state["bias"], state["residual"], act=c["act"],
                                     out_dtype=state["out"])}
    return _plain_moe(state, c) if c["op"] == "moe" else _plain_linear(state, c)


# ---- work --------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        rows = 2 * N if c["act"] == "swiglu" else N
        size = {"none": 0, "bf16": 2, "f32": 4}
        b = 2 * M * K + 2 * rows * K + (4 * rows if c["bias"] else 0) + M * N * (size[c["residual"]] + size[c["out"]])
        return {"bytes": b, "flops": 2 * M * rows * K}
    T, H, E, k, I = c["T"], c["H"], c["E"], c["k"], c["I"]
    g = 2 if c["act"] == "swiglu" else 1
    # bytes of one weight: 4-bit codes with two bf16 per 64, or one byte per 16
    per = {"bf16": 2.0, "affine4": 0.5 + 4 / 64, "nvfp4": 0.5 + 1 / 16}[c["fmt"]]
    active = E * (1 - (1 - k / E) ** T)                  # experts that T tokens pick between them
    rows = (g + 1) * H * (active * I + c["Is"])
    b = per * rows + 4 * E * H + 4 * E + 2 * T * H * (2 + bool(c["residual"])) + 8 * T * k
    return {"bytes": int(b), "flops": int(2 * T * (g + 1) * H * (k * I + c["Is"]) + 2 * T * E * H)}


# ---- the 64-bit value --------------------------------------------------------
def _value(W, fmt, e):
    """One expert's weights as float64, a nibble at a time."""
    w = W["w"][e]
    if fmt == "bf16":
        return w.double()
    if fmt == "affine4":
        out = torch.empty((w.shape[0], w.shape[1] * 8), dtype=torch.float64, device=w.device)
        for i in range(8):
            out[:, i::8] = torch.bitwise_and(torch.bitwise_right_shift(w, 4 * i), 15).double()
        rep = out.shape[1] // W["scale"].shape[-1]
        return out * W["scale"][e].double().repeat_interleave(rep, 1) + W["bias"][e].double().repeat_interleave(rep, 1)
    out = torch.empty((w.shape[0], w.shape[1] * 2), dtype=torch.float64, device=w.device)
    for i in range(2):
        code = torch.bitwise_and(torch.bitwise_right_shift(w.int(), 4 * i), 15)
        mag, ex = torch.bitwise_and(code, 1).double(), torch.bitwise_and(torch.bitwise_right_shift(code, 1), 3)
        v = torch.where(ex == 0, mag * 0.5, (1 + mag * 0.5) * 2.0 ** (ex.double() - 1))
        out[:, i::2] = torch.where(code >= 8, -v, v)
    sc = W["scale"][e].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    return out * sc * W["glob"][e].double()


def _ffn(x, w1, w2, c):
    z = w1 @ x
    if c["act"] == "relu2":
        h = torch.where(z > 0, z * z, torch.zeros_like(z))
    else:
        n = z.shape[0] // 2
        g, u = z[:n], z[n:]
        if c["limit"]:
            g, u = torch.minimum(g, torch.full_like(g, c["limit"])), u.clamp(-c["limit"], c["limit"])
        h = g * torch.sigmoid(g) * u
    return w2 @ h


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "linear":
        z = torch.empty((c["M"], s["w"].shape[0]), dtype=torch.float64, device=DEV)
        wt = s["w"].double().t().contiguous()
        for a in range(0, c["M"], 1024):
            z[a:a + 1024] = s["x"][a:a + 1024].double() @ wt
        if c["bias"]:
            z += s["bias"].double()
        if c["act"] == "relu2":
            z = torch.where(z > 0, z * z, torch.zeros_like(z))
        elif c["act"] == "swiglu":
            z = z[:, :c["N"]] * torch.sigmoid(z[:, :c["N"]]) * z[:, c["N"]:]
        if s["residual"] is not None:
            z = z + s["residual"].double()
        return {"y": z}
    x = s["x"].double()
    logits = (x[:, None, :] * s["wr"].double()[None]).sum(-1)
    score = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, -1)
    rank = (score + s["eb"].double()).cpu().tolist()
    idx = [sorted(range(c["E"]), key=lambda e: (-row[e], e))[:c["k"]] for row in rank]
    pick = torch.tensor(idx, device=DEV)
    w = score.gather(1, pick)
    if c["norm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-6)
    y = torch.zeros_like(x)
    for e in sorted({e for row in idx for e in row}):
        w1, w2 = _value(s["W1"], c["fmt"], e), _value(s["W2"], c["fmt"], e)
        for t, row in enumerate(idx):
            if e in row:
                y[t] += w[t, row.index(e)] * _ffn(x[t], w1, w2, c)
    y *= c["out_scale"]
    if c["Is"]:
        w1, w2 = _value(s["S1"], c["fmt"], 0), _value(s["S2"], c["fmt"], 0)
        for t in range(c["T"]):
            y[t] += _ffn(x[t], w1, w2, c)
    if s["residual"] is not None:
        y += s["residual"].double()
    return {"y": y, "idx": pick.int(), "w": w}
