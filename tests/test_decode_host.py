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
