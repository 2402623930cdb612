"""moe_decode refuses bad arguments on the host, before anything is launched.
Fake pointer values are never dereferenced: every call fails validation first."""
import ctypes

import pytest

from sigmoid_top_routing_b200 import abi


@pytest.fixture(scope="module")
def lib():
    from sigmoid_top_routing_b200 import build
    build.build(quiet=True)
    return abi.load()


def _d(T=4, H=256, E=8, k=2, I=128):
    return abi.moe_dims(T, H, E, k, I)


def _w(**over):
    return abi.moe_experts_w(**{**dict(fmt=0, act=0, w1=0x100000, w2=0x200000), **over})


def _layer(W=None, Ws=None, Is=0, score=0, norm=1, w_router=0x50000, bias=None):
    return abi.moe_layer(w_router, bias, W or _w(), Ws or abi.moe_experts_w(), Is, 1e-6, 1.0, 1.0,
                         abi.moe_router_cfg(score, norm))


def _call(lib, L=None, d=None, **over):
    d = d or _d()
    a = dict(x=0x10000, logits=None, residual=None, idx=0x20000, w=0x30000, y=0x40000, ws=0x1000000, n=1 << 24)
    a.update(over)
    st = lib.moe_decode(ctypes.byref(L or _layer()), ctypes.byref(d), a["x"], a["logits"], a["residual"], a["idx"],
                        a["w"], a["y"], a["ws"], a["n"], None)
    if st != abi.MOE_OK:
        assert lib.moe_last_error()
    return st


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=17), dict(T=16, H=4160), dict(H=100), dict(I=96), dict(E=257),
                                 dict(k=9), dict(T=5, H=16384)])
def test_sizes(lib, bad):
    assert _call(lib, d=_d(**bad)) == abi.MOE_ERR_SHAPE
    assert lib.moe_decode_workspace_bytes(ctypes.byref(_d(**bad)), 0) == 0


@pytest.mark.parametrize("Is", [-64, 32, 16448])
def test_shared_width(lib, Is):
    assert _call(lib, _layer(Ws=_w(), Is=Is)) == abi.MOE_ERR_SHAPE


def test_workspace(lib):
    d = _d(T=16, H=4096, E=256, k=32, I=2048)
    n = lib.moe_decode_workspace_bytes(ctypes.byref(d), 1024)
    assert n % 256 == 0 and n >= 1024 + 16 * 256 * 8 + 16 * 32 * 2048 * 2 + 16 * 1024 * 2
    L = _layer(Ws=_w(), Is=1024)
    assert _call(lib, L, d, n=n - 1) == abi.MOE_ERR_WORKSPACE
    assert _call(lib, L, d, ws=None) == abi.MOE_ERR_WORKSPACE
    assert _call(lib, L, d, ws=0x1000080) == abi.MOE_ERR_ALIGN


@pytest.mark.parametrize("over,status", [
    (dict(x=None), abi.MOE_ERR_NULL), (dict(y=None), abi.MOE_ERR_NULL), (dict(idx=None), abi.MOE_ERR_NULL),
    (dict(w=None), abi.MOE_ERR_NULL), (dict(x=0x10008), abi.MOE_ERR_ALIGN), (dict(y=0x40002), abi.MOE_ERR_ALIGN),
    (dict(residual=0x60008), abi.MOE_ERR_ALIGN), (dict(logits=0x60002), abi.MOE_ERR_ALIGN),
    (dict(idx=0x20002), abi.MOE_ERR_ALIGN),
    (dict(residual=0x40200), abi.MOE_ERR_UNSUPPORTED), (dict(residual=0x40000 - 2032), abi.MOE_ERR_UNSUPPORTED),
])
def test_pointers(lib, over, status):
    assert _call(lib, **over) == status


@pytest.mark.parametrize("layer,status", [
    (dict(w_router=None), abi.MOE_ERR_NULL), (dict(w_router=0x50004), abi.MOE_ERR_ALIGN),
    (dict(score=2), abi.MOE_ERR_UNSUPPORTED), (dict(norm=2), abi.MOE_ERR_UNSUPPORTED),
    (dict(W=_w(fmt=7)), abi.MOE_ERR_UNSUPPORTED), (dict(W=_w(act=2)), abi.MOE_ERR_UNSUPPORTED),
    (dict(W=_w(w1=None)), abi.MOE_ERR_NULL), (dict(W=_w(fmt=1)), abi.MOE_ERR_NULL),
    (dict(W=_w(fmt=2)), abi.MOE_ERR_NULL), (dict(W=_w(swiglu_limit=-1.0)), abi.MOE_ERR_SHAPE),
    (dict(Ws=_w(act=1), Is=64), abi.MOE_ERR_UNSUPPORTED), (dict(Ws=_w(w2=None), Is=64), abi.MOE_ERR_NULL),
])
def test_layer(lib, layer, status):
    assert _call(lib, _layer(**layer)) == status


def test_prepared_plan(lib):
    """What prepare refuses, run never sees; run refuses anything that is no plan."""
    plan = abi.moe_decode_plan()
    assert lib.moe_decode_prepare(ctypes.byref(_layer()), ctypes.byref(_d(T=17)), ctypes.byref(plan)) == abi.MOE_ERR_SHAPE
    assert lib.moe_decode_prepare(ctypes.byref(_layer()), ctypes.byref(_d()), None) == abi.MOE_ERR_NULL
    args = (0x10000, None, None, 0x20000, 0x30000, 0x40000, 0x1000000, 1 << 24, None)
    assert lib.moe_decode_run(None, *args) == abi.MOE_ERR_NULL
    assert lib.moe_decode_run(ctypes.byref(plan), *args) == abi.MOE_ERR_UNSUPPORTED


def test_null_layer_and_empty_batch(lib):
    assert lib.moe_decode(None, ctypes.byref(_d()), 0x10000, None, None, 0x20000, 0x30000, 0x40000, 0x1000000, 1 << 24,
                          None) == abi.MOE_ERR_NULL
    assert _call(lib, d=_d(T=0), x=None, y=None, ws=None) == abi.MOE_OK
    assert lib.moe_last_launch_count() == 0


def test_python_layer_refuses_cpu_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    from sigmoid_top_routing_b200 import api
    W = api.ExpertWeights(act=0, fmt=0, w1=torch.zeros(4, 128, 64, dtype=torch.bfloat16),
                          w2=torch.zeros(4, 64, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        api.DecodeLayer(W, torch.zeros(4, 64), E=4, k=2, I=64)


# ---- shared-memory layout of the weight ring ----------------------------------
SMEM = 232448                                          # 227 KB, the most a CTA of the device may have
ROWS = [64, 192, 256, 320, 512, 704, 1024, 1472, 1856, 1984, 2048, 2112, 2240, 2304, 2560, 2688, 3008, 3712, 4096,
        4160, 7168, 8128, 8192, 16320, 16384]
HIDDEN = [64, 320, 2048, 2176, 2688, 4096, 16384]


def _layouts(lib, fmt):
    """(layout, T, H, I, Is) of every combination of the sizes above that is allowed."""
    for T in range(1, 17):
        for H in HIDDEN:
            if T * H > 65536:
                continue
            for I in ROWS:
                for Is in [0] + ROWS:
                    m, d = abi.moe_decode_smem(), _d(T=T, H=H, I=I)
                    assert lib.moe_decode_smem_layout(ctypes.byref(d), Is, fmt, SMEM, ctypes.byref(m)) == abi.MOE_OK
                    if m.smem:
                        yield m, T, H, I, Is


def _scales_of(fmt, K):
    """Bytes of one scale array of K weights."""
    return K // 32 if fmt == abi.MOE_W_AFFINE4_G64 else K // 16


def _copies(fmt, st, K, boxed):
    """(offset from the array's start, most bytes) of the scale copies of a stage of rows of K."""
    if boxed:
        return [(h * (st.area // 2), 8 * (64 if fmt == abi.MOE_W_AFFINE4_G64 else 128)) for h in range(2)]
    if K <= 2048:                                      # 8 rows' span, widened to 16-byte units
        return [(h * (st.area // 2), (8 * _scales_of(fmt, K) + 30) // 16 * 16) for h in range(2)]
    return [(r * st.area / 16, (_scales_of(fmt, min(st.k, K)) + 30) // 16 * 16) for r in range(16)]


def _check_stage(m, fmt, st, rows, tokens, where):
    """Every copy of a stage starts on 16 bytes, has room, and touches no other."""
    arrays = 0 if fmt == abi.MOE_W_BF16 else 2 if fmt == abi.MOE_W_AFFINE4_G64 else 1
    assert st.scales == 2 * st.half == 2048 * st.chunks, where
    assert st.tokens == st.scales + arrays * st.area and st.tokens % 16 == 0, where
    pad = 64 if fmt == abi.MOE_W_BF16 else 16
    assert st.tokens + tokens * (2 * st.k + pad) <= st.bytes <= m.stage_bytes, where
    for K, boxed in rows:
        for a in range(arrays):
            copies = _copies(fmt, st, K, boxed)
            ends = [o for o, _ in copies[1:]] + [st.area]
            for (o, n), end in zip(copies, ends):
                assert o == int(o) and (st.scales + a * st.area + int(o)) % 16 == 0, (where, K, o)
                assert o + n <= end, (where, K, o, n, end)


@pytest.mark.parametrize("fmt", [abi.MOE_W_BF16, abi.MOE_W_AFFINE4_G64, abi.MOE_W_NVFP4])
def test_every_copy_of_a_stage_is_aligned_and_inside(lib, fmt):
    seen = 0
    for m, T, H, I, Is in _layouts(lib, fmt):
        where = (T, H, I, Is)
        assert m.stage_bytes % 1024 == 0 and m.slots >= 1, where
        assert (m.ring + 1023) // 1024 * 1024 + 4 * m.slots * m.stage_bytes <= m.smem <= SMEM, where
        _check_stage(m, fmt, m.up, [(H, m.boxed_up)], 0, where)
        down = [(I, m.boxed_down)] + ([(Is, m.boxed_shared)] if Is else [])
        _check_stage(m, fmt, m.down, down, T, where)
        seen += 1
    assert seen > 50000


def test_layout_refusals(lib):
    m = abi.moe_decode_smem()
    call = lib.moe_decode_smem_layout
    assert call(ctypes.byref(_d(T=17)), 0, 0, SMEM, ctypes.byref(m)) == abi.MOE_ERR_SHAPE
    assert call(ctypes.byref(_d(T=0)), 0, 0, SMEM, ctypes.byref(m)) == abi.MOE_ERR_SHAPE
    assert call(ctypes.byref(_d()), 32, 0, SMEM, ctypes.byref(m)) == abi.MOE_ERR_SHAPE
    assert call(ctypes.byref(_d()), 0, 3, SMEM, ctypes.byref(m)) == abi.MOE_ERR_UNSUPPORTED
    assert call(ctypes.byref(_d()), 0, 0, SMEM, None) == abi.MOE_ERR_NULL
    assert call(ctypes.byref(_d()), 0, 0, 1024, ctypes.byref(m)) == abi.MOE_OK and m.smem == 0


@pytest.mark.parametrize("fmt,period", [(abi.MOE_W_AFFINE4_G64, 512), (abi.MOE_W_NVFP4, 1024)])
def test_boxed_scales_start_on_their_swizzle_period(lib, fmt, period):
    """TMA swizzles by address bits: a box off its period has its rows' 16-byte units elsewhere."""
    boxes = 0
    for m, T, H, I, Is in _layouts(lib, fmt):
        for st, boxed in ((m.up, m.boxed_up), (m.down, m.boxed_down or m.boxed_shared)):
            if boxed:
                arrays = 2 if fmt == abi.MOE_W_AFFINE4_G64 else 1
                starts = [st.scales + a * st.area + h * (st.area // 2) for a in range(arrays) for h in range(2)]
                assert all(s % period == 0 for s in starts), (T, H, I, Is, st.scales, st.area)
                boxes += 1
    assert boxes > 50000


@pytest.mark.parametrize("polls", [0, (1 << 20) + 1])
def test_expiry_check_refuses_its_polls(lib, polls):
    plan = abi.moe_decode_plan()
    args = (0x10000, None, None, 0x20000, 0x30000, 0x40000, 0x1000000, 1 << 24)
    assert lib.moe_decode_expiry_check(ctypes.byref(plan), *args, polls, None) == abi.MOE_ERR_SHAPE
    assert lib.moe_decode_expiry_check(ctypes.byref(plan), *args, 1, None) == abi.MOE_ERR_UNSUPPORTED   # no plan
    assert lib.moe_decode_expiry_check(None, *args, 1, None) == abi.MOE_ERR_NULL


# T = 4, H = 256, E = 8, k = 2: x, residual and y are 2048 bytes, logits 128, picks 32
@pytest.mark.parametrize("over", [
    dict(idx=0x10000), dict(idx=0x10000 + 2044), dict(w=0x10000 - 28), dict(residual=0x60000, w=0x60400),
    dict(logits=0x60000, idx=0x60000), dict(logits=0x60000, w=0x60000 + 124), dict(idx=0x30000), dict(w=0x20000 + 28),
    dict(w=0x40000), dict(idx=0x40000 + 2044), dict(idx=0x40000 - 28), dict(y=0x1000000), dict(w=0x1000100),
])
def test_picks_over_other_arguments(lib, over):
    assert _call(lib, **over) == abi.MOE_ERR_UNSUPPORTED
    assert b"overlaps" in lib.moe_last_error()
