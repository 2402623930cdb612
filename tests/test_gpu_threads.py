"""Calls from threads that have not used the device: the first thing such a thread does
may be any call of the library.  (Outputs are allocated beforehand: an allocation in
the thread could make the device's context current by itself.)"""
import threading

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


@pytest.fixture(scope="module")
def block():
    from sigmoid_top_routing_b200 import inputs as G
    from sigmoid_top_routing_b200.device_inputs import to_device
    wl = G.Workload("threads", T=16, H=512, E=8, k=2, I=128)
    return wl, to_device(G.make_inputs(wl))


def in_new_threads(n, f):
    """f(i) in n new threads at once; whatever they raise."""
    raised = []

    def run(i):
        try:
            f(i)
        except BaseException as e:  # noqa: BLE001
            raised.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if raised:
        raise raised[0]


@pytest.mark.parametrize("M", [8, 2000])
def test_linear(api, M):
    x, w = torch.randn(M, 256, device="cuda").bfloat16(), torch.randn(512, 256, device="cuda").bfloat16()
    want = api.moe_linear(x, w)
    y = [torch.zeros_like(want) for _ in range(4)]
    torch.cuda.synchronize()
    in_new_threads(4, lambda i: api.moe_linear(x, w, y=y[i]))
    assert all(torch.equal(t, want) for t in y)


def test_decode_layers_prepare_in_their_threads(api, block):
    """Token counts that a layer has not seen are prepared by the calling thread."""
    wl, D = block
    layers = [api.DecodeLayer(D.W, D.w_router, D.expert_bias, E=wl.E, k=wl.k, I=wl.I) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in layers]
    want = [t.clone() for t in layers[0](D.x)]
    got = [[] for _ in layers]
    torch.cuda.synchronize()

    def work(i):
        for T in (3, 9, 1, 16, 5):
            with torch.cuda.stream(streams[i]):
                got[i].append(layers[i](D.x[:T]))
    in_new_threads(4, work)
    for outs in got:
        assert len(outs) == 5
        for out in outs:
            for a, b in zip(out, want):
                assert torch.equal(a, b[:len(a)])


def test_experts(api, block):
    """The grouped GEMM of 16 tokens reads x itself: its tensor maps come before its first launch."""
    wl, D = block
    kw = dict(E=wl.E, I=wl.I)
    idx, w = api.moe_route(D.x, None, D.w_router, D.expert_bias, E=wl.E, k=wl.k)
    plan = api.moe_plan(idx, E=wl.E, H=wl.H, I=wl.I)
    want = api.moe_experts(D.x, plan, w, D.W, combine=1, dispatch=2, **kw)
    d = api.dims(wl.T, wl.H, wl.E, wl.k, wl.I)
    ws = [api.new_workspace(d, dispatch=2, combine=1) for _ in range(2)]
    y = [torch.zeros_like(want) for _ in range(2)]
    torch.cuda.synchronize()
    in_new_threads(2, lambda i: api.moe_experts(D.x, plan, w, D.W, combine=1, dispatch=2, y=y[i], ws=ws[i], **kw))
    assert all(torch.equal(t, want) for t in y)
