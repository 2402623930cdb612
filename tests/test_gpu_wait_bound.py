"""Failure detection on the GPU without a fault: the tcgen05 pipelines'
bounded mbarrier wait is made to run out on purpose (a barrier nothing
arrives on, a short poll limit, in a one-warp kernel with no TMA and no TMEM),
and the host reads the error code it leaves; the context stays usable, which
a normal forward right after shows by passing oracle parity."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def api():
    from sigmoid_top_routing_b200 import build
    build.build(quiet=True)
    from sigmoid_top_routing_b200 import api as A
    A.load()
    return A


def test_expired_wait_reports_code_2_and_context_survives(api):
    from sigmoid_top_routing_b200 import abi, inputs
    from sigmoid_top_routing_b200.device_inputs import to_device
    lib = api.load()
    assert api.moe_device_error() == 0                      # start clean
    assert lib.moe_wait_bound_check(4096, None) == abi.MOE_OK
    assert api.moe_device_error() == 2                      # the wait ran out and said so
    assert api.moe_device_error() == 0                      # read-and-clear
    assert lib.moe_wait_bound_check(0, None) == abi.MOE_ERR_SHAPE
    assert lib.moe_wait_bound_check((1 << 20) + 1, None) == abi.MOE_ERR_SHAPE

    wl = inputs.WORKLOADS["lfm2_decode_t8"]
    inp = inputs.make_inputs(wl)
    D = to_device(inp)
    y, idx, w, _ = api.moe_forward(D.x, D.W, D.w_router, D.expert_bias, E=wl.E, k=wl.k, I=wl.I, eps=wl.eps,
                                   dispatch=abi.MOE_DISPATCH_GEMM)
    torch.cuda.synchronize()
    assert api.moe_device_error() == 0
    ref = oracle.moe_block(inp)
    assert np.array_equal(idx.cpu().numpy(), ref["idx"])
    yg = y.float().cpu().numpy().astype(np.float64)
    assert np.linalg.norm(yg - ref["y"]) / np.linalg.norm(ref["y"]) < 1e-2


@pytest.mark.parametrize("polls", [1, 4096])
@pytest.mark.parametrize("fmt,T,shared_I,given", [("bf16", 8, 0, False), ("bf16", 2, 128, True), ("affine4", 9, 320, False),
                                                  ("nvfp4", 16, 64, False), ("nvfp4", 1, 0, True)])
def test_decode_layer_whose_grid_barriers_run_out(api, fmt, T, shared_I, given, polls):
    """The call records error 2 and ends, y keeps its bytes, and the next call with the
    same workspace has the same bits as before."""
    import ctypes

    from sigmoid_top_routing_b200 import abi, inputs
    from sigmoid_top_routing_b200.device_inputs import shared_to_device, to_device
    wl = inputs.Workload("expiry", T=T, H=320, E=24, k=5, I=704, fmt=fmt, shared_I=shared_I)
    inp = inputs.make_inputs(wl)
    D, Ws = to_device(inp), shared_to_device(inp)
    layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, E=wl.E, k=wl.k, I=wl.I, Ws=Ws, Is=shared_I)
    logits = torch.randn(T, wl.E, device="cuda") if given else None
    want = [t.clone() for t in layer(D.x, logits=logits)]
    G = torch.cuda.get_device_properties(0).multi_processor_count
    y = torch.full_like(want[0], 7.0)
    idx, w = torch.empty_like(want[1]), torch.empty_like(want[2])
    for _ in range(2):
        st = api.load().moe_decode_expiry_check(
            layer._plans[T][1], D.x.data_ptr(), None if logits is None else logits.data_ptr(), None, idx.data_ptr(),
            w.data_ptr(), y.data_ptr(), layer.ws.data_ptr(), layer.ws.numel(), polls,
            torch.cuda.current_stream().cuda_stream)
        assert st == abi.MOE_OK
        torch.cuda.synchronize()
        assert api.moe_device_error() == 2
        assert (y == 7.0).all()
        assert int(layer.ws[:8].view(torch.int64)) % G == 0 and (layer.ws[8:1024] == 0).all()
        for a, b in zip(layer(D.x, logits=logits), want):
            assert torch.equal(a, b)
        assert api.moe_device_error() == 0


@pytest.mark.parametrize("polls", [1, 4096])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("M,N,K", [(3, 200, 64), (8, 2048, 2048), (40, 5000, 1000), (130, 300, 300),   # one CTA or a cluster a tile
                                   (700, 2048, 1024), (4096, 2048, 64), (2000, 1100, 5000)])           # SM pairs
def test_linear_layer_whose_wait_runs_out(api, M, N, K, act, polls):
    """The call records error 2 and ends, y keeps its bytes, and the next call is right."""
    import ctypes

    from sigmoid_top_routing_b200 import abi
    rows, ld = (2 * N if act == "swiglu" else N), (K + 7) // 8 * 8
    x = torch.randn(M, ld, device="cuda").bfloat16()[:, :K]
    w = (torch.randn(rows, ld, device="cuda") * K ** -0.5).bfloat16()[:, :K]
    want = api.moe_linear(x, w, act=act)
    y = torch.full_like(want, 7.0)
    d = abi.moe_linear_dims(M, N, K, ld, ld, 0, 0)
    c = abi.moe_linear_cfg(abi.MOE_ACT_SWIGLU if act == "swiglu" else abi.MOE_ACT_NONE, 0, 0, 0.0)
    for _ in range(2):
        st = api.load().moe_linear_expiry_check(x.data_ptr(), w.data_ptr(), None, None, ctypes.byref(d), ctypes.byref(c),
                                                y.data_ptr(), polls, torch.cuda.current_stream().cuda_stream)
        assert st == abi.MOE_OK
        torch.cuda.synchronize()
        assert api.moe_device_error() == 2
        assert (y == 7.0).all()
        assert torch.equal(api.moe_linear(x, w, act=act), want)
        assert api.moe_device_error() == 0
