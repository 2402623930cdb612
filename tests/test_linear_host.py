"""moe_linear refuses bad arguments on the host, before anything is launched
(fake pointers, never dereferenced), and its Python wrapper checks shapes, types
and strides."""
import ctypes

import pytest

from sigmoid_top_routing_b200 import abi


@pytest.fixture(scope="module")
def lib():
    from sigmoid_top_routing_b200 import build
    build.build(quiet=True)
    return abi.load()


def _call(lib, *, M=4, N=32, K=64, ldx=0, ldw=0, ldr=0, ldy=0, act=2, res_f32=0, y_f32=0, limit=0.0, x=0x10000,
          w=0x20000, bias=None, residual=None, y=0x30000):
    d, c = abi.moe_linear_dims(M, N, K, ldx, ldw, ldr, ldy), abi.moe_linear_cfg(act, res_f32, y_f32, limit)
    st = lib.moe_linear(x, w, bias, residual, ctypes.byref(d), ctypes.byref(c), y, None)
    if st != abi.MOE_OK:
        assert lib.moe_last_error()
    return st


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), abi.MOE_ERR_SHAPE), (dict(N=0), abi.MOE_ERR_SHAPE), (dict(K=0), abi.MOE_ERR_SHAPE),
    (dict(K=(1 << 24) + 1), abi.MOE_ERR_SHAPE), (dict(ldx=56), abi.MOE_ERR_SHAPE), (dict(ldy=31), abi.MOE_ERR_SHAPE),
    (dict(ldr=31), abi.MOE_ERR_SHAPE), (dict(ldw=-8), abi.MOE_ERR_SHAPE), (dict(K=63), abi.MOE_ERR_ALIGN),
    (dict(ldx=68), abi.MOE_ERR_ALIGN), (dict(ldw=66), abi.MOE_ERR_ALIGN), (dict(act=3), abi.MOE_ERR_UNSUPPORTED),
    (dict(res_f32=2), abi.MOE_ERR_UNSUPPORTED), (dict(y_f32=-1), abi.MOE_ERR_UNSUPPORTED),
    (dict(limit=-1.0), abi.MOE_ERR_SHAPE), (dict(limit=float("nan")), abi.MOE_ERR_SHAPE),
    (dict(limit=float("inf")), abi.MOE_ERR_SHAPE), (dict(x=None), abi.MOE_ERR_NULL), (dict(w=None), abi.MOE_ERR_NULL),
    (dict(y=None), abi.MOE_ERR_NULL), (dict(x=0x10008), abi.MOE_ERR_ALIGN), (dict(w=0x20004), abi.MOE_ERR_ALIGN),
    (dict(bias=0x40002), abi.MOE_ERR_ALIGN), (dict(y=0x30001), abi.MOE_ERR_ALIGN),
    (dict(y=0x30002, y_f32=1), abi.MOE_ERR_ALIGN), (dict(residual=0x50002, res_f32=1), abi.MOE_ERR_ALIGN),
])
def test_refusals(lib, bad, status):
    assert _call(lib, **bad) == status


# M = 4, N = 32, K = 64 at their dense strides: x is 512 bytes, w 4096, bias 128, y 256
@pytest.mark.parametrize("bad", [
    dict(y=0x10000), dict(y=0x101fe), dict(y=0x10000 - 254), dict(y=0x20000 + 4094), dict(act=0, y=0x20000 + 8190),
    dict(bias=0x30000), dict(bias=0x30000 - 124), dict(act=0, bias=0x30000 - 252),
    dict(residual=0x30040), dict(residual=0x30000, res_f32=1), dict(residual=0x30000, ldr=40),
    dict(x=0x10000, ldx=128, y=0x1007e, ldy=128),                    # column blocks that share column 63
    dict(x=0x10000, ldx=128, y=0x10080 + 66, ldy=128),               # a block that runs into the next row of x
    dict(x=0x10000, ldx=128, y=0x10080, ldy=64),                     # interleaved with another stride
    dict(M=1, x=0x10000, y=0x10010),
    dict(M=1, y=0x20000 + 128 * 5),                                  # a single row of y in w
])
def test_outputs_over_inputs(lib, bad):
    assert _call(lib, **bad) == abi.MOE_ERR_UNSUPPORTED


def test_null_structs_and_empty_batch(lib):
    c = abi.moe_linear_cfg(2, 0, 0, 0.0)
    assert lib.moe_linear(0x10000, 0x20000, None, None, None, ctypes.byref(c), 0x30000, None) == abi.MOE_ERR_NULL
    assert _call(lib, M=0, x=None, y=None) == abi.MOE_OK
    assert lib.moe_last_launch_count() == 0


def test_python_wrapper_needs_cuda():
    torch = pytest.importorskip("torch")
    from sigmoid_top_routing_b200 import api
    with pytest.raises(ValueError):
        api.moe_linear(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16))


@pytest.mark.parametrize("polls", [0, (1 << 20) + 1])
def test_expiry_check_refuses_its_polls(lib, polls):
    d, c = abi.moe_linear_dims(4, 32, 64, 0, 0, 0, 0), abi.moe_linear_cfg(2, 0, 0, 0.0)
    call = lib.moe_linear_expiry_check
    assert call(0x10000, 0x20000, None, None, ctypes.byref(d), ctypes.byref(c), 0x30000, polls, None) == abi.MOE_ERR_SHAPE
    assert call(0x10000, 0x20000, None, None, ctypes.byref(d), ctypes.byref(c), None, 1, None) == abi.MOE_ERR_NULL
