"""The few-token MoE layer (moe_decode) against the float64 oracle.

Tolerances.  A rounding to bf16 is off by at most u = 2^-8 of the value.  The
kernel rounds twice: every activation h to bf16, and y.  So per element
    |y_gpu - y| <= u |y| + u A (1 + s),   A = out_scale sum_j |w_j| sum_i |W2| |h| + the shared expert's,
where s covers the fp32 sums: a pre-activation is off by at most n 2^-24 of its
sum of absolute products (n = H terms), which in units of u is below 1 for the
sizes here (H <= 4096: 4096 * 2^-24 = u / 16 of that sum; |act'| of it enters h).
s = 1 is used.  The norm-wise gate: errors of independent roundings, each at
most u relative, leave at most sqrt(2) u of y's norm when nothing cancels
systematically; 2 u is the gate.  Picks must be the oracle's; weights are
float64 rounded once to fp32 (2^-24; 2^-23 allows for exp's own last bit).
"""
import dataclasses

import numpy as np
import pytest

import oracle as O
from sigmoid_top_routing_b200 import inputs as G

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -8


@pytest.fixture(scope="module")
def api():
    from sigmoid_top_routing_b200 import build
    build.build(quiet=True)
    from sigmoid_top_routing_b200 import api as A
    A.load()
    return A


_CACHE = {}


def inputs_of(wl):
    if wl not in _CACHE:
        _CACHE.clear()
        _CACHE[wl] = G.make_inputs(wl)
    return _CACHE[wl]


def residual_of(wl):
    r = np.random.default_rng(7).standard_normal((wl.T, wl.H)).astype(np.float32)
    return G.f32_to_bf16_bits(r)


def make_layer(api, inp, **over):
    from sigmoid_top_routing_b200.device_inputs import shared_to_device, to_device
    wl = inp.wl
    D = to_device(inp)
    kw = dict(E=wl.E, k=wl.k, I=wl.I, Ws=shared_to_device(inp), Is=wl.shared_I, eps=wl.eps,
              router_scale=wl.router_scale, out_scale=wl.out_scale, score=wl.score, norm_topk=wl.norm_topk,
              max_tokens=wl.T)
    kw.update(over)
    layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, **kw)
    layer.ws[1024:].fill_(0xFF)                      # only the counts need zeros
    return D, layer


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def magnitude(inp, r):
    """A of the module docstring, for every element of y."""
    wl = inp.wl
    x = O.bf16_to_f64(inp.x_bits)
    A = np.zeros((wl.T, wl.H))
    from oracle.moe_oracle import _act, _expert_w, _shared_w
    for e in np.unique(r["idx"]):
        W1, W2 = _expert_w(inp, "w1", int(e)), _expert_w(inp, "w2", int(e))
        for t, j in zip(*np.nonzero(r["idx"] == e)):
            h = _act(x[t:t + 1] @ W1.T, wl.act, wl.I, wl.swiglu_limit)
            A[t] += abs(r["w"][t, j]) * (np.abs(h) @ np.abs(W2).T)[0]
    A *= abs(wl.out_scale)
    if wl.shared_I:
        h = _act(x @ _shared_w(inp, "w1").T, wl.act, wl.shared_I, wl.swiglu_limit)
        A += np.abs(h) @ np.abs(_shared_w(inp, "w2")).T
    return A


def compare(inp, y, idx, w, residual=None, logits=None):
    r = O.moe_block(inp, use_logits=logits)
    nan = np.isnan(r["c"]).all(axis=1)
    assert np.array_equal(idx, r["idx"])
    np.testing.assert_allclose(w[~nan], r["w"][~nan], rtol=2.0 ** -23, atol=0)
    want = r["y"] + (O.bf16_to_f64(residual) if residual is not None else 0.0)
    got = O.bf16_to_f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want).any(axis=1)
    if ok.any():
        err = np.abs(got - want)[ok]
        tol = U * np.abs(want) + 2 * U * magnitude(inp, r)
        assert (err <= tol[ok] + 1e-30).all(), (err / (tol[ok] + 1e-30)).max()
        # the norm of what the experts add, not of the residual
        assert np.linalg.norm(err) <= 2 * U * np.linalg.norm(want[ok])


def run_and_compare(api, wl, residual=True, logits=None):
    inp = inputs_of(wl)
    D, layer = make_layer(api, inp)
    res = residual_of(wl) if residual else None
    from sigmoid_top_routing_b200.device_inputs import bf16_tensor
    rt = bf16_tensor(res, "cuda") if residual else None
    # outputs inside guard rows: nothing outside them is written
    yb = torch.full((wl.T + 2, wl.H), -1, dtype=torch.int16, device="cuda")
    ib = torch.full((wl.T + 2, wl.k), -1, dtype=torch.int32, device="cuda")
    wb = torch.full((wl.T + 2, wl.k), -1, dtype=torch.int32, device="cuda")
    y = yb.view(torch.bfloat16)[1:-1]
    lg = None if logits is None else torch.from_numpy(logits).cuda()
    layer(D.x, residual=rt, logits=lg, y=y, topk_idx=ib[1:-1], topk_w=wb.view(torch.float32)[1:-1])
    torch.cuda.synchronize()
    assert api.moe_device_error() == 0
    assert api.moe_last_launch_count() == 1
    for b in (yb, ib, wb):
        assert (b[0] == -1).all() and (b[-1] == -1).all()
    G = torch.cuda.get_device_properties(0).multi_processor_count
    assert int(layer.ws[:8].view(torch.int64)) % G == 0 and (layer.ws[8:1024] == 0).all()
    compare(inp, bits(y), ib[1:-1].cpu().numpy(), wb.view(torch.float32)[1:-1].cpu().numpy(), res, logits)


W = G.Workload


@pytest.mark.parametrize("fmt", ["bf16", "affine4", "nvfp4"])
@pytest.mark.parametrize("wl", [
    W("one", T=1, H=64, E=1, k=1, I=64),                                       # the smallest sizes
    W("tiny", T=3, H=256, E=8, k=2, I=128, swiglu_limit=1.0),
    W("relu2", T=5, H=320, E=16, k=6, I=192, act="relu2", out_scale=2.5),      # 3 groups: odd scale rows
    W("shared", T=8, H=448, E=12, k=3, I=320, shared_I=576, out_scale=0.5),
    W("wide", T=9, H=2176, E=6, k=2, I=192, shared_I=64),                      # 9 columns; 4-bit rows in 2 chunks
    W("long", T=2, H=192, E=4, k=2, I=4160, act="relu2"),                      # long down rows, odd groups
    W("many", T=16, H=128, E=256, k=32, I=64),                                 # the most experts and picks
    W("few_rows", T=9, H=320, E=24, k=5, I=704, shared_I=256, out_scale=0.5),  # blocks of y shared by CTAs
    W("two_blocks", T=16, H=1152, E=40, k=2, I=256, act="relu2"),
    W("softmax", T=13, H=512, E=40, k=5, I=256, score="softmax", norm_topk=False),
], ids=lambda w: w.name)
def test_parity(api, wl, fmt):
    run_and_compare(api, dataclasses.replace(wl, fmt=fmt, name=f"{wl.name}_{fmt}"))


@pytest.mark.parametrize("fmt", ["bf16", "affine4", "nvfp4"])
def test_limits_of_the_sizes(api, fmt):
    run_and_compare(api, W("t16", T=16, H=4096, E=4, k=2, I=64, shared_I=64, fmt=fmt))   # T * H = 65536
    run_and_compare(api, W("t15", T=15, H=4352, E=3, k=1, I=128, act="relu2", fmt=fmt))


def test_longest_rows(api):
    run_and_compare(api, W("h16384", T=4, H=16384, E=3, k=1, I=64), residual=False)


@pytest.mark.parametrize("fmt", ["bf16", "affine4", "nvfp4"])
def test_one_expert_takes_every_token(api, fmt):
    """Two column blocks of one expert, the others empty."""
    wl = W("hot", T=16, H=256, E=8, k=1, I=192, fmt=fmt)
    lg = np.full((16, 8), -4.0, dtype=np.float32)
    lg[:, 3] = 4.0
    run_and_compare(api, wl, logits=lg)


def test_ties_take_the_lower_expert(api):
    wl = W("ties", T=4, H=128, E=40, k=7, I=64, score="softmax")
    lg = np.zeros((4, 40), dtype=np.float32)
    lg[1, 35:] = 1.0
    lg[2, ::2] = -0.0
    inp = inputs_of(wl)
    inp.expert_bias[:] = 0.0
    run_and_compare(api, wl, logits=lg)
    _CACHE.clear()


@pytest.mark.parametrize("T,E,k", [(3, 12, 4), (16, 200, 6)])                 # ranked by counting, and by rounds
def test_close_scores_rank_by_their_64_bit_values(api, T, E, k):
    """Logits one fp32 step apart: their fp32 sigmoids are equal, their real ones are not."""
    wl = W("close", T=T, H=64, E=E, k=k, I=64)
    inp = inputs_of(wl)
    inp.expert_bias[:] = 0.0
    lg = np.full((T, E), -3.0, dtype=np.float32)
    v = np.float32(9.0)
    for i in range(k + 2):                                                     # the larger, the later its expert
        lg[:, E - 2 * (k + 2) + 2 * i] = v
        v = np.nextafter(v, np.float32(20.0))
    s32 = (1 / (1 + np.exp(-lg[0]))).astype(np.float32)
    assert len(np.unique(s32)) == 2                                            # one value but for the -3s
    run_and_compare(api, wl, residual=False, logits=lg)
    _CACHE.clear()


def test_router_sums_survive_cancellation(api):
    """Expert logits of ~1e-3 apart that are differences of terms of ~1e4: an fp32 sum
    would not rank them."""
    wl = W("cancel", T=5, H=512, E=16, k=3, I=64)
    inp = inputs_of(wl)
    rng = np.random.default_rng(4)
    x = O.bf16_to_f64(inp.x_bits)
    x[:, 256:] = -x[:, :256]                                                   # exact in bf16
    inp.x_bits[:] = G.f32_to_bf16_bits(x.astype(np.float32))
    big = (rng.standard_normal((16, 256)) * 1e4).astype(np.float32)
    small = (rng.standard_normal((16, 256)) * 1e-3).astype(np.float32)
    inp.w_router[:] = np.concatenate([big + small, big], axis=1)
    want = x @ inp.w_router.astype(np.float64).T
    seq = np.zeros((5, 16), dtype=np.float32)
    for h in range(512):
        seq += x[:, h:h + 1].astype(np.float32) * inp.w_router[None, :, h]
    assert np.abs(seq - want).max() > 1e-3                                     # what one fp32 chain would give
    run_and_compare(api, wl)
    _CACHE.clear()


def test_one_shot_c_call(api):
    """moe_decode is moe_decode_prepare and moe_decode_run in one."""
    import ctypes

    from sigmoid_top_routing_b200 import abi
    wl = W("oneshot", T=6, H=256, E=8, k=2, I=128, shared_I=64)
    D, layer = make_layer(api, inputs_of(wl))
    want, idx, w = layer(D.x)
    y, i2, w2 = torch.empty_like(want), torch.empty_like(idx), torch.empty_like(w)
    d = abi.moe_dims(wl.T, wl.H, wl.E, wl.k, wl.I)
    st = abi.load().moe_decode(ctypes.byref(layer._layer), ctypes.byref(d), D.x.data_ptr(), None, None, i2.data_ptr(),
                               w2.data_ptr(), y.data_ptr(), layer.ws.data_ptr(), layer.ws.numel(),
                               torch.cuda.current_stream().cuda_stream)
    assert st == abi.MOE_OK
    assert torch.equal(y, want) and torch.equal(i2, idx) and torch.equal(w2, w)


def test_layers_share_a_workspace_in_turn(api):
    """Layers of other sizes may take turns on one zeroed workspace."""
    a = make_layer(api, G.make_inputs(W("ws_a", T=9, H=320, E=24, k=5, I=704)))
    b = make_layer(api, G.make_inputs(W("ws_b", T=2, H=256, E=8, k=2, I=128, fmt="nvfp4")))
    want = [[t.clone() for t in layer(D.x)] for D, layer in (a, b)]
    ws = torch.zeros(max(a[1].ws.numel(), b[1].ws.numel()), dtype=torch.uint8, device="cuda")
    a[1].ws = b[1].ws = ws
    for _ in range(3):
        for (D, layer), ref in zip((a, b), want):
            for t, r in zip(layer(D.x), ref):
                assert torch.equal(t, r)


def test_calls_on_two_streams_of_two_layers(api):
    """Layers of their own may be called at once."""
    made = [make_layer(api, G.make_inputs(W(f"par{i}", T=4, H=512, E=16, k=4, I=256, seed=i))) for i in range(2)]
    want = [[t.clone() for t in layer(D.x)] for D, layer in made]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (D, layer) in enumerate(made):
            with torch.cuda.stream(streams[i]):
                got[i].append(layer(D.x, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            for t, r in zip(out, want[i]):
                assert torch.equal(t, r)


def test_nan_and_infinite_rows(api):
    """A row of NaN picks 0..k-1 and its output is NaN; its neighbours do not notice."""
    wl = W("nan", T=6, H=256, E=8, k=3, I=128, nan_rows=2)
    run_and_compare(api, wl)
    wl = dataclasses.replace(wl, name="inf", nan_rows=0)
    lg = np.random.default_rng(3).standard_normal((6, 8)).astype(np.float32)
    lg[1] = np.nan
    lg[2, 4] = np.nan
    lg[3, 5] = np.inf
    lg[4, :] = -np.inf
    run_and_compare(api, wl, logits=lg)


@pytest.mark.parametrize("alias", ["residual", "x"])
def test_output_in_place(api, alias):
    wl = W("alias", T=7, H=320, E=8, k=2, I=128, shared_I=64)
    inp = inputs_of(wl)
    D, layer = make_layer(api, inp)
    from sigmoid_top_routing_b200.device_inputs import bf16_tensor
    r = bf16_tensor(residual_of(wl), "cuda")
    want, idx, w = layer(D.x, residual=r)
    dst = r if alias == "residual" else D.x
    got, idx2, w2 = layer(D.x, residual=r, y=dst)
    assert torch.equal(got, want) and torch.equal(idx, idx2) and torch.equal(w, w2)
    assert got.data_ptr() == dst.data_ptr()


def test_empty_batch(api):
    wl = W("empty", T=2, H=64, E=2, k=1, I=64)
    D, layer = make_layer(api, inputs_of(wl))
    y, idx, w = layer(D.x[:0])
    assert y.shape == (0, 64) and idx.shape == (0, 1) and api.moe_last_launch_count() == 0


def test_fewer_tokens_than_max_and_repeated_calls(api):
    """One workspace serves every T up to max_tokens, call after call, with the same bits."""
    wl = W("rep", T=16, H=512, E=16, k=4, I=256, shared_I=128)
    D, layer = make_layer(api, inputs_of(wl))
    first = {T: layer(D.x[:T]) for T in (16, 1, 8, 9, 3)}
    for T in (3, 9, 8, 1, 16):
        for a, b in zip(first[T], layer(D.x[:T])):
            assert torch.equal(a, b)


def test_graph_and_side_stream(api):
    wl = W("graph", T=4, H=512, E=16, k=4, I=256)
    D, layer = make_layer(api, inputs_of(wl))
    x = D.x.clone()
    want = [t.clone() for t in layer(x)]
    x2 = (D.x.float() * 0.5).bfloat16()
    want2 = [t.clone() for t in layer(x2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer(x)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(x)
        out2 = layer(out[0], residual=x)
    for src, ref in ((D.x, want), (x2, want2), (D.x, want)):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, out):
            assert torch.equal(a, b)
        for a, b in zip(layer(ref[0], residual=src), out2):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["lfm2_decode_t8", "affine4_t8", "nvfp4_t1", "affine4_t1"])
def test_agrees_with_moe_forward(api, name):
    """The layer and the multi-kernel block: same picks, outputs within both sides' roundings."""
    wl = G.WORKLOADS[name]
    inp = inputs_of(wl)
    D, layer = make_layer(api, inp)
    y, idx, w = layer(D.x)
    y2, idx2, w2, _ = api.moe_forward(D.x, D.W, D.w_router, D.expert_bias, E=wl.E, k=wl.k, I=wl.I, eps=wl.eps,
                                      router_scale=wl.router_scale, out_scale=wl.out_scale)
    assert torch.equal(idx, idx2)
    a, b = y.float(), y2.float()
    assert (a - b).norm() <= 4 * U * b.norm()
    compare(inp, bits(y), idx.cpu().numpy(), w.cpu().numpy())


def test_python_refusals(api):
    wl = W("refuse", T=4, H=128, E=4, k=2, I=64)
    D, layer = make_layer(api, inputs_of(wl))
    with pytest.raises(ValueError):
        layer(torch.cat([D.x, D.x]))                             # more than max_tokens
    with pytest.raises(ValueError):
        layer(D.x.float())
    with pytest.raises(ValueError):
        layer(D.x[:, ::2])
    with pytest.raises(ValueError):
        layer(D.x, residual=D.x[:2])
    with pytest.raises(ValueError):
        layer(D.x.cpu())
    with pytest.raises(ValueError):
        api.DecodeLayer(D.W, D.w_router, D.expert_bias, E=4, k=2, I=128)
    with pytest.raises(ValueError):
        api.DecodeLayer(D.W, D.w_router, D.expert_bias, E=4, k=2, I=64, max_tokens=17)


# A down stage serves w2 and the shared w2; their scale rows lie differently when one
# of I, Is is above 2048 and the other is not.  Without a residual, so that the norm
# gate sees what the experts add.
@pytest.mark.parametrize("fmt", ["affine4", "nvfp4"])
@pytest.mark.parametrize("wl", [
    W("wide_shared_t4", T=4, H=2688, E=6, k=3, I=1856, act="relu2", shared_I=3712),
    W("wide_shared_t16", T=16, H=2688, E=6, k=3, I=1856, act="relu2", shared_I=3712, out_scale=2.5),
    W("wide_shared_t10", T=10, H=320, E=8, k=2, I=1984, shared_I=2112),
    W("wide_experts_t7", T=7, H=448, E=5, k=2, I=2240, shared_I=1472),
    W("wide_experts_t15", T=15, H=4096, E=3, k=1, I=4160, shared_I=64, act="relu2"),
], ids=lambda w: w.name)
def test_shared_width_across_2048(api, wl, fmt):
    run_and_compare(api, dataclasses.replace(wl, fmt=fmt, name=f"{wl.name}_{fmt}"), residual=False)


# NVFP4: one of the two scale arrays in swizzled boxes, the other in row slots, in the
# same stage; y in blocks of more than 8 rows, whose second half reads the second box.
@pytest.mark.parametrize("wl", [
    W("box_i_t1", T=1, H=2048, E=4, k=2, I=2048, shared_I=2112),
    W("box_is_t1", T=1, H=2176, E=4, k=2, I=2112, shared_I=256, act="relu2"),
    W("box_i_t2", T=2, H=256, E=6, k=3, I=1536, shared_I=3008),
    W("box_is_t2", T=2, H=2048, E=4, k=2, I=2240, shared_I=2048, out_scale=0.5),
    W("box_long_t5", T=5, H=2432, E=3, k=2, I=4096, shared_I=2496, act="relu2"),
], ids=lambda w: w.name)
def test_boxed_and_slotted_scales_in_one_stage(api, wl):
    run_and_compare(api, dataclasses.replace(wl, fmt="nvfp4"), residual=False)


@pytest.mark.parametrize("E", [16, 200])                                       # ranked by counting, and by rounds
def test_softmax_ranks_large_logits_by_their_64_bit_values(api, E):
    """Router logits of tens of thousands: rounded to fp32 they move a softmax score by
    5e-5, far past the distance at which two fp32 scores count as close.  The expert bias
    sets the scores 4e-5 apart; the tokens share them and differ in a common shift of
    their logits."""
    T, k, n = 16, 5, 12                                                        # n experts in the running
    wl = W("soft_large", T=T, H=256, E=E, k=k, I=64, score="softmax")
    inp = inputs_of(wl)
    rng = np.random.default_rng(0)
    x = np.repeat(O.bf16_to_f64(inp.x_bits)[:1], T, axis=0)
    x[:, 0] = 200 + 2 * np.arange(T)
    inp.x_bits[:] = G.f32_to_bf16_bits(x.astype(np.float32))
    inp.w_router[:, 1:] *= 1.5
    inp.w_router[:, 0] = 125.0
    runners = rng.permutation(E)[:n]
    out = np.setdiff1d(np.arange(E), runners)
    inp.w_router[out, 0] = 123.0                                               # 64 and more behind: a score of ~0
    L = O.bf16_to_f64(inp.x_bits) @ inp.w_router.astype(np.float64).T

    def softmax(v):
        p = np.exp(v - v.max(axis=1, keepdims=True))
        return p / p.sum(axis=1, keepdims=True)
    p = softmax(L)
    inp.expert_bias[:] = -1.0
    inp.expert_bias[runners] = (0.3 - p[0, runners] + 4e-5 * rng.permutation(n)).astype(np.float32)
    want = np.argsort(-(p + inp.expert_bias), axis=1)[:, :k]
    r = softmax(L.astype(np.float32).astype(np.float64)) + inp.expert_bias     # scores of rounded logits
    order = np.argsort(-r, axis=1)[:, :k + 1]
    c = np.take_along_axis(r, order, axis=1)
    far = (c[:, :-1] - c[:, 1:] > 4e-6 * (1 + c[:, :-1])).all(axis=1)
    assert (far & (order[:, :k] != want).any(axis=1)).sum() >= 4               # wrong, and no two of them close
    run_and_compare(api, wl, residual=False)
    _CACHE.clear()


@pytest.mark.parametrize("fmt", ["bf16", "affine4", "nvfp4"])
def test_layer_keeps_the_tensors_it_was_given(api, fmt):
    """Fields of the weights set to other tensors, and the router dropped, after the layer was made."""
    import gc
    import weakref

    from sigmoid_top_routing_b200.device_inputs import shared_to_device, to_device
    wl = W("keep", T=4, H=256, E=8, k=2, I=128, shared_I=64, fmt=fmt)
    inp = inputs_of(wl)
    D, Ws = to_device(inp), shared_to_device(inp)
    layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, E=wl.E, k=wl.k, I=wl.I, Ws=Ws, Is=wl.shared_I)
    want = [t.clone() for t in layer(D.x)]
    refs, shapes = [weakref.ref(D.w_router), weakref.ref(D.expert_bias)], []
    for w in (D.W, Ws):
        for f in dataclasses.fields(w):
            t = getattr(w, f.name)
            if isinstance(t, torch.Tensor):
                refs.append(weakref.ref(t))
                shapes.append((t.shape, t.dtype))
                setattr(w, f.name, None)
                del t
    x = D.x
    del D, Ws, w
    gc.collect()
    assert all(r() is not None for r in refs)
    junk = [torch.empty(s, dtype=d, device="cuda").view(torch.uint8).fill_(0xFF) for s, d in shapes]
    for T in (4, 3):                                          # 3: prepared after the change
        for a, b in zip(layer(x[:T]), want):
            assert torch.equal(a, b[:T])
    del junk


def comparable_residual(wl, ref_y):
    """bf16 residual of about the experts' own size (a power of two times N(0, 1)): an
    error of their sum is not drowned by the residual's own rounding."""
    rms = np.sqrt(np.mean(ref_y ** 2))
    r = np.random.default_rng(9).standard_normal((wl.T, wl.H)) * 2.0 ** np.round(np.log2(rms))
    return G.f32_to_bf16_bits(r.astype(np.float32))


def strict_gate(got, ref_y, residual=None):
    """Norm of the error against the roundings': y's, at most U of what is stored, and the
    activations', whose independent relative errors of at most U each reach at most U of
    the experts' sum when it does not cancel systematically."""
    want = ref_y + (O.bf16_to_f64(residual) if residual is not None else 0.0)
    err, gate = np.linalg.norm(got - want), U * (np.linalg.norm(want) + np.linalg.norm(ref_y))
    assert err <= gate, err / gate


def test_the_gate_sees_a_missing_or_scaled_part():
    """The gate on the oracle's own values: a twentieth too little, or no residual, fails it."""
    ref = np.random.default_rng(1).standard_normal((8, 256)) * 1e-3
    wl = W("gate", T=8, H=256, E=1, k=1, I=64)
    r = comparable_residual(wl, ref)
    full = ref + O.bf16_to_f64(r)
    strict_gate(full, ref, r)
    for bad in (ref, O.bf16_to_f64(r), full - 0.05 * ref):
        with pytest.raises(AssertionError):
            strict_gate(bad, ref, r)
    with pytest.raises(AssertionError):
        strict_gate(0.97 * ref, ref)


@pytest.mark.parametrize("fmt", ["bf16", "affine4", "nvfp4"])
@pytest.mark.parametrize("wl", next(m.args[1] for m in test_parity.pytestmark if m.args[0] == "wl"), ids=lambda w: w.name)
def test_experts_alone_and_beside_a_residual_of_their_size(api, wl, fmt):
    inp = inputs_of(dataclasses.replace(wl, fmt=fmt, name=f"{wl.name}_{fmt}"))
    D, layer = make_layer(api, inp)
    from sigmoid_top_routing_b200.device_inputs import bf16_tensor
    ref = O.moe_block(inp)
    res = comparable_residual(wl, ref["y"])
    for r in (None, res):
        y, idx, w = layer(D.x, residual=None if r is None else bf16_tensor(r, "cuda"))
        compare(inp, bits(y), idx.cpu().numpy(), w.cpu().numpy(), r)
        strict_gate(O.bf16_to_f64(bits(y)), ref["y"], r)
