"""moe_linear against the formula in float64.

Tolerances.  A pre-activation v is an fp32 sum of K products of bf16 values
(each exact in fp32): off by at most d = (K + 1) 2^-23 S, S = sum |x w| + |b|
(2^-23: a sum may be truncated rather than rounded).  Through the activation
  none    d
  relu^2  2 |v| d + d^2 + 2^-23 v^2
  swiglu  |u| 1.1 dg + |silu(g)| du + dg du + 2^-21 |silu(g) u|   (|silu'| < 1.1; exp, divide, product)
then one fp32 addition of the residual (2^-24) and the store's rounding, 2^-8 of
the value for bf16.  These worst cases are far above what happens, so the norm is
gated too: independent errors of each of K additions give 2^-23 sqrt(K) of the
norm (times 2 through the square and the gate's product), the store 2^-8.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def api():
    from sigmoid_top_routing_b200 import build
    build.build(quiet=True)
    from sigmoid_top_routing_b200 import api as A
    A.load()
    return A


def silu(g):
    return g * torch.sigmoid(g)


def formula(x, w, bias, residual, act, limit, y_dtype):
    """(value, bound on the error) in float64."""
    X, Wd = x.double(), w.double()
    K = X.shape[1]
    v, S = X @ Wd.t(), X.abs() @ Wd.abs().t()
    if bias is not None:
        v, S = v + bias.double(), S + bias.double().abs()
    d = (K + 1) * 2.0 ** -23 * S
    if act == "none":
        o, tol = v, d
    elif act == "relu2":
        o = v.clamp_min(0) ** 2
        tol = 2 * v.abs() * d + d * d + 2.0 ** -23 * v * v
    else:
        N = v.shape[1] // 2
        g, u, dg, du = v[:, :N], v[:, N:], d[:, :N], d[:, N:]
        if limit > 0:
            g, u = g.clamp_max(limit), u.clamp(-limit, limit)
        o = silu(g) * u
        tol = u.abs() * 1.1 * dg + silu(g).abs() * du + dg * du + 2.0 ** -21 * o.abs()
    if residual is not None:
        o = o + residual.double()
        tol = tol + 2.0 ** -24 * o.abs()
    if y_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (o.abs() + tol)
    return o, tol + 2.0 ** -126


def make(M, N, K, act="none", bias=False, residual=None, seed=0, ldpad=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rows = 2 * N if act == "swiglu" else N
    ld = (K + 7) // 8 * 8 + ldpad

    def mat(r, c, scale):
        t = torch.full((r, c), float("nan"), device="cuda").bfloat16()      # pads that must not be read
        t[:, :K] = torch.randn((r, K), generator=gen, device="cuda") * scale
        return t[:, :K]
    x, w = mat(M, ld, 1.0), mat(rows, ld, 1.0 / math.sqrt(K))
    b = torch.randn(rows, generator=gen, device="cuda") if bias else None
    r = torch.randn((M, N), generator=gen, device="cuda").to(residual) if residual is not None else None
    return x, w, b, r


def check(api, x, w, b, r, act="none", limit=0.0, out=torch.bfloat16, y=None):
    K = x.shape[1]
    want, tol = formula(x, w, b, r, act, limit, out)
    got = api.moe_linear(x, w, b, r, act=act, swiglu_limit=limit, out_dtype=out, y=y)
    torch.cuda.synchronize()
    assert api.moe_device_error() == 0 and api.moe_last_launch_count() == 1
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), float((err / tol).max())
    gate = 2 * 2.0 ** -23 * math.sqrt(K + 1) + (2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -23)
    assert err.norm() <= gate * want.norm().clamp_min(1e-30), float(err.norm() / want.norm())
    return got


SIZES = [(1, 1, 1), (1, 2048, 2048), (2, 7, 8), (5, 64, 63), (15, 130, 65), (16, 1, 200), (17, 257, 1795),
         (33, 1537, 64), (77, 96, 4096), (128, 129, 24), (129, 64, 512), (300, 700, 136), (511, 2049, 321),
         (1000, 2100, 200), (4096, 33, 72), (70, 20000, 48)]


@pytest.mark.parametrize("act", ["none", "relu2", "swiglu"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(api, M, N, K, act):
    x, w, b, r = make(M, N, K, act, bias=True, residual=torch.bfloat16)
    check(api, x, w, b, r, act)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [3, 640])
def test_types(api, M, bias, res, out):
    for act in ("none", "swiglu"):
        x, w, b, r = make(M, 1100, 264, act, bias=bias, residual=res, seed=M)
        check(api, x, w, b, r, act, out=out)


@pytest.mark.parametrize("M", [9, 900])
def test_strides_and_guards(api, M):
    """Wider rows of x and w (their pads hold NaN), residual and y inside wider
    buffers at odd offsets; what lies around y keeps its bytes."""
    N, K = 1031, 333
    x, w, b, _ = make(M, N, K, bias=True, ldpad=24)
    rb = torch.randn((M, N + 5), device="cuda").bfloat16()
    yb = torch.full((M + 2, N + 7), 7.5, device="cuda")
    y = yb[1:-1, 3:3 + N]
    got = check(api, x, w, b, rb[:, 5:], out=torch.float32, y=y)
    assert got.data_ptr() == y.data_ptr()
    keep = torch.ones_like(yb, dtype=torch.bool)
    keep[1:-1, 3:3 + N] = False
    assert (yb[keep] == 7.5).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [8, 700])
def test_residual_in_place(api, M, dtype):
    x, w, b, r = make(M, 1500, 256, bias=True, residual=dtype)
    want = api.moe_linear(x, w, b, r, out_dtype=dtype)
    got = api.moe_linear(x, w, b, r, y=r)
    assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("M", [1, 6, 700])
def test_column_blocks_of_one_buffer(api, M):
    """x, the residual and y side by side in the rows of one buffer."""
    x, w, b, r = make(M, 64, 256, bias=True, residual=torch.bfloat16)
    buf = torch.full((M, 400), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, :256], buf[:, 264:328] = x, r
    check(api, buf[:, :256], w, b, buf[:, 264:328], y=buf[:, 328:392])
    assert torch.equal(buf[:, :256], x) and torch.equal(buf[:, 264:328], r)
    assert buf[:, 256:264].isnan().all() and buf[:, 392:].isnan().all()
    with pytest.raises(RuntimeError, match="overlaps"):
        api.moe_linear(buf[:, :256], w, b, y=buf[:, 192:256])
    with pytest.raises(RuntimeError, match="overlaps"):
        api.moe_linear(x, w, b, buf[:, 328:392], y=buf[:, 330:394])


@pytest.mark.parametrize("M", [4, 512])
def test_clamp_and_special_values(api, M):
    x, w, b, r = make(M, 600, 128, "swiglu", bias=True, seed=5)
    check(api, x * 4, w, b, r, "swiglu", limit=1.5)
    x, w, b, _ = make(M, 600, 128, "relu2", bias=True)
    x = x.clone()
    x[1] = float("nan")
    x[2, 3] = float("inf")
    w = w.clone()
    w[:, 3] = w[:, 3].abs() + 0.01
    y = api.moe_linear(x, w, b, act="relu2")
    assert torch.isnan(y[1]).all() and torch.isinf(y[2]).all()
    rows = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(y[rows], api.moe_linear(x[rows].contiguous(), w, b, act="relu2")) or M > 64
    assert torch.isfinite(y[rows]).all()
    w2 = w.clone()
    w2[5] = float("nan")                              # one feature's weights: one column of y
    y = api.moe_linear(x[3:4], w2, b, act="none")
    assert torch.isnan(y[:, 5]).all() and torch.isfinite(y[:, 6:]).all() and torch.isfinite(y[:, :5]).all()


@pytest.mark.parametrize("M", [1, 40, 2000])
def test_reproducible_graph_and_side_stream(api, M):
    x, w, b, r = make(M, 1024, 1024, "swiglu", bias=True, residual=torch.float32)
    first = api.moe_linear(x, w, b, r, act="swiglu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = [api.moe_linear(x, w, b, r, act="swiglu") for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    for y in again:
        assert torch.equal(y, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h = api.moe_linear(x, w, b, r, act="swiglu")
        z = api.moe_linear(h, w[:1024], residual=h)
    x2 = x.clone()
    for scale in (1.0, -0.5):
        x.copy_(x2 * scale)
        g.replay()
        torch.cuda.synchronize()
        want = api.moe_linear(x, w, b, r, act="swiglu")
        assert torch.equal(h, want)
        assert torch.equal(z, api.moe_linear(want, w[:1024], residual=want))


def test_empty_batch(api):
    x, w, b, _ = make(4, 64, 64)
    assert api.moe_linear(x[:0], w).shape == (0, 64)
    assert api.moe_last_launch_count() == 0


def test_python_refusals(api):
    x, w, b, r = make(4, 64, 64, bias=True, residual=torch.bfloat16)
    bad = [dict(x=x.float()), dict(w=w[:, :32]), dict(w=w.cpu()), dict(bias=b[:10]), dict(bias=b.bfloat16()),
           dict(residual=r[:2]), dict(residual=r.half()), dict(y=torch.empty(4, 63, device="cuda")), dict(act="gelu"),
           dict(x=x.t().contiguous().t()), dict(act="swiglu", w=w[:63]),
           dict(y=torch.empty(4, 64, device="cuda"), out_dtype=torch.bfloat16), dict(x=x[0])]
    for over in bad:
        kw = dict(x=x, w=w, bias=b, residual=r)
        kw.update(over)
        with pytest.raises(ValueError):
            api.moe_linear(kw.pop("x"), kw.pop("w"), **kw)
    big = torch.zeros(4, 66, device="cuda").bfloat16()
    with pytest.raises(api.abi.MoEError):
        api.moe_linear(big[:, :64], w)                # rows of x start off 16 bytes


def test_layers_of_a_hybrid_stack(api):
    """Dense relu^2 layer, dense SwiGLU layer and a sparse layer with a shared expert
    in a row, as a decode step runs them, against float64 with the same roundings
    between the layers; the shared expert also as two moe_linear calls."""
    import numpy as np

    import oracle as O
    from sigmoid_top_routing_b200 import inputs as G
    from sigmoid_top_routing_b200.device_inputs import shared_to_device, to_device
    wl = G.Workload("stack", T=6, H=512, E=16, k=3, I=192, shared_I=320, out_scale=1.5)
    inp = G.make_inputs(wl)
    D, Ws = to_device(inp), shared_to_device(inp)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)

    def mat(n, k):
        return (torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)).bfloat16()
    up, down, gate_up, down2 = mat(1024, 512), mat(512, 1024), mat(2 * 768, 512), mat(512, 768)
    x = D.x
    h = api.moe_linear(x, up, act="relu2")
    x1 = api.moe_linear(h, down, residual=x)
    h = api.moe_linear(x1, gate_up, act="swiglu")
    x2 = api.moe_linear(h, down2, residual=x1)
    layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, E=wl.E, k=wl.k, I=wl.I, Ws=Ws, Is=wl.shared_I,
                            out_scale=wl.out_scale)
    y, idx, w = layer(x2, residual=x2)
    # the linear layers, each from its own rounded input
    for xin, w1, w2, act, out in ((x, up, down, "relu2", x1), (x1, gate_up, down2, "swiglu", x2)):
        hid, _ = formula(xin, w1, None, None, act, 0.0, torch.bfloat16)
        want = hid.bfloat16().double() @ w2.double().t() + xin.double()
        # two bf16 roundings: the hidden values' (2^-8, through w2 at most its norm) and the result's
        assert (out.double() - want).norm() <= 2 * 2.0 ** -8 * want.norm()
    inp2 = G.make_inputs(wl)
    inp2.x_bits = x2.view(torch.int16).cpu().numpy().view(np.uint16)
    ref = O.moe_block(inp2)
    assert np.array_equal(idx.cpu().numpy(), ref["idx"])
    want = torch.from_numpy(ref["y"]).cuda() + x2.double()
    assert (y.double() - want).norm() <= 2 * 2.0 ** -8 * want.norm()
    # the shared expert as two linear layers, into moe_forward's y_shared
    hs = api.moe_linear(x2, Ws.w1[0], act="swiglu")
    y_shared = api.moe_linear(hs, Ws.w2[0], out_dtype=torch.float32)
    y2, idx2, _, _ = api.moe_forward(x2, D.W, D.w_router, D.expert_bias, E=wl.E, k=wl.k, I=wl.I,
                                     out_scale=wl.out_scale, y_shared=y_shared)
    assert torch.equal(idx, idx2)
    moe = torch.from_numpy(ref["y"]).cuda()
    assert (y2.double() - moe).norm() <= 3 * 2.0 ** -8 * moe.norm()   # h and hs rounded, then y


@pytest.mark.parametrize("M,act", [(4, "relu2"), (512, "relu2"), (512, "swiglu"), (512, "none"), (2000, "relu2")])
def test_rows_beside_nan_and_infinite_rows(api, M, act):
    """Tokens whose tile also holds a NaN and an infinite token keep to the formula's bound."""
    x, w, b, r = make(M, 600, 128, act, bias=True, residual=torch.bfloat16, seed=6)
    x = x.clone()
    x[1] = float("nan")
    x[2, 3] = float("inf")
    y = api.moe_linear(x, w, b, r, act=act)
    rows = [i for i in range(M) if i not in (1, 2)]
    want, tol = formula(x[rows], w, b, r[rows], act, 0.0, torch.bfloat16)
    assert torch.isnan(y[1]).all()
    assert ((y[rows].double() - want).abs() <= tol).all()


def test_more_than_2_to_the_31_elements(api):
    """Offsets of y and of the residual past 32 bits, in place."""
    M, N, K = 600_000, 4096, 64
    x, w, b, _ = make(M, N, K, bias=True)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda").normal_()
    rows = torch.tensor([0, 1, 262_143, 262_144, 524_287, 524_288, 599_999], device="cuda")   # 2^30 elements and multiples
    want, tol = formula(x[rows], w, b, y[rows], "none", 0.0, torch.bfloat16)
    api.moe_linear(x, w, b, y, y=y)
    assert ((y[rows].double() - want).abs() <= tol).all()
