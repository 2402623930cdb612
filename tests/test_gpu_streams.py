"""Calls with ``stream=`` another stream than the current one: what the wrapper
allocates belongs to the stream that writes it, so a block that the current stream
still writes is not handed out.  Every test enqueues, on the current stream, a wait
and then a write into a block that it frees at once."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CYCLES = 100_000_000                                   # ~50 ms: longer than any call here


@pytest.fixture(scope="module")
def api():
    from sigmoid_top_routing_b200 import build
    build.build(quiet=True)
    from sigmoid_top_routing_b200 import api as A
    A.load()
    return A


@pytest.fixture(scope="module")
def block():
    """(workload, device inputs) of a small block."""
    from sigmoid_top_routing_b200 import inputs as G
    from sigmoid_top_routing_b200.device_inputs import to_device
    wl = G.Workload("streams", T=8, H=512, E=8, k=2, I=128)
    return wl, to_device(G.make_inputs(wl))


def freed_but_written_later(*shapes):
    """Blocks of the outputs' sizes that the current stream writes after a while, freed now."""
    torch.cuda._sleep(CYCLES)
    for shape, dtype in shapes:
        for _ in range(4):
            torch.empty(shape, dtype=dtype, device="cuda").view(torch.uint8).fill_(0x55)


def same(got, want):
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("raw", [False, True])
def test_linear(api, raw):
    x, w = torch.randn(64, 256, device="cuda").bfloat16(), torch.randn(512, 256, device="cuda").bfloat16()
    want = api.moe_linear(x, w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed_but_written_later(((64, 512), torch.bfloat16))
    same([api.moe_linear(x, w, stream=s.cuda_stream if raw else s)], [want])


def test_decode_layer(api, block):
    wl, D = block
    layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, E=wl.E, k=wl.k, I=wl.I)
    want = [t.clone() for t in layer(D.x)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed_but_written_later(((wl.T, wl.H), torch.bfloat16), ((wl.T, wl.k), torch.int32))
    same(layer(D.x, stream=s), want)


def test_forward_and_its_parts(api, block):
    wl, D = block
    kw = dict(E=wl.E, k=wl.k, I=wl.I)
    want = [t.clone() for t in api.moe_forward(D.x, D.W, D.w_router, D.expert_bias, combine=1, **kw)[:3]]
    s = torch.cuda.Stream()
    n = api.moe_workspace_bytes(api.dims(wl.T, wl.H, wl.E, wl.k, wl.I), combine=1)
    torch.cuda.synchronize()
    shapes = (((wl.T, wl.H), torch.bfloat16), ((wl.T, wl.k), torch.int32), ((n,), torch.uint8))
    freed_but_written_later(*shapes)
    got = api.moe_forward(D.x, D.W, D.w_router, D.expert_bias, combine=1, stream=s, **kw)
    same(got[:3], want)
    freed_but_written_later(*shapes)
    idx, w = api.moe_route(D.x, None, D.w_router, D.expert_bias, E=wl.E, k=wl.k, stream=s)
    plan = api.moe_plan(idx, E=wl.E, H=wl.H, I=wl.I, stream=s)
    y = api.moe_experts(D.x, plan, w, D.W, E=wl.E, I=wl.I, combine=1, stream=s)
    same([y, idx, w], want)


def test_shared_expert(api, block):
    wl, D = block
    Ws = api.ExpertWeights(act=D.W.act, fmt=D.W.fmt, w1=D.W.w1[:1], w2=D.W.w2[:1])
    want = api.moe_shared_expert(D.x, Ws, I=wl.I, combine=1)
    s = torch.cuda.Stream()
    n = api.moe_workspace_bytes(api.dims(wl.T, wl.H, 1, 1, wl.I), combine=1)
    torch.cuda.synchronize()
    freed_but_written_later(((wl.T, wl.H), torch.float32), ((n,), torch.uint8))
    same([api.moe_shared_expert(D.x, Ws, I=wl.I, combine=1, stream=s)], [want])


def test_layer_made_on_a_busy_stream_and_first_called_on_another(api, block):
    """The workspace's counts are zero whichever stream calls first."""
    wl, D = block
    kw = dict(E=wl.E, k=wl.k, I=wl.I)
    layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, **kw)
    want, n = [t.clone() for t in layer(D.x)], layer.ws.numel()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")     # the block that the workspace will get
        torch.cuda._sleep(CYCLES)
        layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, **kw)
        assert a.query()                                             # zeroed when the constructor returns
    same(layer(D.x, stream=b), want)
    assert api.moe_device_error() == 0


def test_workspace_outlives_its_layer_on_another_stream(api, block):
    """The layer is dropped while a call of it waits on a side stream; its workspace is not handed out."""
    wl, D = block
    kw = dict(E=wl.E, k=wl.k, I=wl.I)
    layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, **kw)
    want = [t.clone() for t in layer(D.x)]
    n, at, s = layer.ws.numel(), layer.ws.data_ptr(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(CYCLES)
    got = layer(D.x, stream=s)
    del layer
    blocks = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert at not in [t.data_ptr() for t in blocks]
    same(got, want)


def replayed(g, out, want):
    for _ in range(3):
        g.replay()
    same(out, want)


def test_first_calls_inside_a_capture(api, block):
    """Token counts that the layer has not seen, a layer made there, and sizes of moe_linear never run before."""
    wl, D = block
    kw = dict(E=wl.E, k=wl.k, I=wl.I)
    want = [t.clone() for t in api.DecodeLayer(D.W, D.w_router, D.expert_bias, **kw)(D.x)]
    layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, **kw)
    w = torch.randn(768, wl.H, device="cuda").bfloat16()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [layer(D.x[:T]) for T in (3, 8)]
        outs.append(api.DecodeLayer(D.W, D.w_router, D.expert_bias, **kw)(D.x[:5]))
        lin = api.moe_linear(D.x, w, act="relu2")
    for out in outs:
        replayed(g, out, [t[:len(out[0])] for t in want])
    same([lin], [api.moe_linear(D.x, w, act="relu2")])
    assert api.moe_device_error() == 0


def test_decode_layer_beside_other_streams_work(api, block):
    """Its launch needs every SM at once; other streams keep them busy."""
    wl, D = block
    layer = api.DecodeLayer(D.W, D.w_router, D.expert_bias, E=wl.E, k=wl.k, I=wl.I)
    x, w = torch.randn(8192, 1024, device="cuda").bfloat16(), torch.randn(2048, 1024, device="cuda").bfloat16()
    want, lin = [t.clone() for t in layer(D.x)], api.moe_linear(x, w)
    a, b, c = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()
    outs, lins = [], []
    for _ in range(20):
        outs.append(layer(D.x, stream=a))
        lins.append(api.moe_linear(x, w, stream=b))
        with torch.cuda.stream(c):
            torch.mm(x, w.t())
    for out in outs:
        same(out, want)
    same(lins, [lin] * len(lins))
    assert api.moe_device_error() == 0


def test_weights_of_another_stream_outlive_their_layer(api, block):
    """Weights allocated on one stream, a layer made and called on a second, then all of it dropped."""
    wl, D = block
    kw = dict(E=wl.E, k=wl.k, I=wl.I)
    want = [t.clone() for t in api.DecodeLayer(D.W, D.w_router, D.expert_bias, **kw)(D.x)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        Wa = D.W.clone()
    a.synchronize()
    at = {Wa.w1.data_ptr(), Wa.w2.data_ptr()}
    shapes = [Wa.w1.shape, Wa.w2.shape]
    with torch.cuda.stream(b):
        layer = api.DecodeLayer(Wa, D.w_router, D.expert_bias, **kw)
        torch.cuda._sleep(CYCLES)
        got = layer(D.x)
    del Wa, layer
    with torch.cuda.stream(a):
        blocks = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in shapes for _ in range(4)]
    assert not at & {t.data_ptr() for t in blocks}
    same(got, want)
