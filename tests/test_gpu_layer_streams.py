"""Layers called on a stream of their own while the current stream is busy: the same results as on the current stream,
for a first call, for a larger one behind it, and for one with a raw handle."""
import numpy as np
import pytest
import torch

from bit_block_quantized_moe_b200 import binding
from gen import CONFIGS, make_layer, make_x

pytestmark = pytest.mark.gpu

BUSY = 400_000_000  # clock cycles: 0.2 s, far more than all calls here together


@pytest.fixture(scope="module")
def M():
    import __graft_entry__

    __graft_entry__.build()
    import bit_block_quantized_moe_b200 as m

    return m


def moe_layer(M, w, cfg):
    return M.Q2MoeLayer(cfg.hidden, cfg.inter, cfg.n_experts, cfg.top_k, w["router_w"], w["router_b"], w["experts"],
                        w["shared"], device="cuda")


def soil(stream):
    """Blocks of every size that the allocator might hand out again on this stream, with foreign bits in them."""
    with torch.cuda.stream(stream):
        held = [torch.full((1 << i,), 0xff, dtype=torch.uint8, device="cuda") for i in range(9, 26)]
    stream.synchronize()
    del held


@pytest.mark.parametrize("raw", [False, True])
def test_moe_layer_on_another_stream(M, raw):
    cfg = CONFIGS["tiny"]
    w = make_layer(cfg, seed=3)
    sizes = (3, 8, 40, 2, 300)
    xs = [torch.from_numpy(np.asarray(make_x(T, cfg.hidden, seed=50 + T)).view(np.int16)).cuda() for T in sizes]
    alone = moe_layer(M, w, cfg)
    want = [alone.forward(x) for x in xs]
    alone.check_status()
    layer, side = moe_layer(M, w, cfg), torch.cuda.Stream()
    out = [torch.empty_like(x) for x in xs]
    soil(side)
    soil(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for x, o in zip(xs, out):
        layer.forward(x, out=o, stream=side.cuda_stream if raw else side)
        # what the allocator has free goes to the current stream's work, which comes later than all calls
        for n in (1 << 10, 1 << 16, 1 << 20, 1 << 22):
            torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # the calls waited for nothing there
    layer.check_status(side)
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_moe_layer_reserved_here_and_called_there(M):
    cfg = CONFIGS["tiny"]
    w = make_layer(cfg, seed=4)
    x = torch.from_numpy(np.asarray(make_x(8, cfg.hidden, seed=1)).view(np.int16)).cuda()
    layer, side = moe_layer(M, w, cfg), torch.cuda.Stream()
    want = layer.forward(x)
    torch.cuda.synchronize()
    layer = moe_layer(M, w, cfg)
    out = torch.empty_like(x)
    soil(torch.cuda.current_stream())
    torch.cuda._sleep(BUSY)
    layer.reserve(8)
    layer.forward(x, out=out, stream=side)
    side.synchronize()
    layer.check_status(side)
    assert torch.equal(out, want)
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        layer.forward(x, out=out)
    layer.reserve(100)  # the old workspace is in use there until this returns
    assert side.query()
    layer.forward(x, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


# ---- the decoder layer ---------------------------------------------------------------------------------------------
def decoder_calls(layer, stream, clean):
    """A prompt and windows of two sequences, each call larger than the buffers of the last or smaller: the residuals,
    next inputs and the cache."""
    import bit_block_quantized_moe_b200 as M

    g = torch.Generator(device="cuda").manual_seed(17)
    hidden, lens, steps = layer.moe.dims.hidden, [600, 2500], []
    for s, n in enumerate(lens):
        layer.cache.grow(s, n)
    layer.cache.k.normal_(generator=g)
    layer.cache.v.normal_(generator=g)
    for m in (1, 3, 40, 2, 200):  # the first one takes parts of a cut group, whose counts have to be zero
        resid = torch.randn((2 * m, hidden), generator=g, device="cuda")
        x = torch.empty((2 * m, hidden), dtype=torch.bfloat16, device="cuda")
        M.moe_rmsnorm_residual(resid, None, x, 2 * m, hidden, 1e-6)
        steps.append((x, resid, torch.empty_like(x)))
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = layer.cache.table(range(2))
    torch.cuda.synchronize()
    clean()
    for x, resid, x_next in steps:
        layer.forward(x, resid, x_next, kv_len, table, stream=stream)
        for n in (1 << 10, 1 << 16, 1 << 20, 1 << 22):
            torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    return [t for _, a, b in steps for t in (a, b)] + [layer.cache.k, layer.cache.v]


@pytest.mark.parametrize("raw", [False, True])
def test_decoder_layer_on_another_stream(M, raw):
    from test_gpu_decoder_layer import build

    alone = build(M, seed=2, pages=200)
    want = decoder_calls(alone, None, lambda: None)
    alone.check_status()
    layer, side = build(M, seed=2, pages=200), torch.cuda.Stream()

    def busy():
        soil(side)
        soil(torch.cuda.current_stream())
        torch.cuda._sleep(BUSY)

    got = decoder_calls(layer, side.cuda_stream if raw else side, busy)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # the calls waited for nothing there
    layer.check_status(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_decoder_layer_reserved_here_and_called_there(M):
    from test_gpu_decoder_layer import build

    want = decoder_calls(build(M, seed=2, pages=200), None, lambda: None)
    layer, side = build(M, seed=2, pages=200), torch.cuda.Stream()

    def reserve():
        soil(torch.cuda.current_stream())
        torch.cuda._sleep(BUSY)
        layer.reserve(400, 2)

    got = decoder_calls(layer, side, reserve)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_decoder_layer_captured_on_a_stream_that_is_not_current(M):
    """The larger call after the capture leaves the graph its buffers, though the capturing stream was only an argument."""
    from test_gpu_decoder_layer import build

    layer, side = build(M, seed=5), torch.cuda.Stream()
    hidden = layer.moe.dims.hidden
    g = torch.Generator(device="cuda").manual_seed(3)
    layer.cache.grow(0, 300)
    table = layer.cache.table([0])
    start = torch.randn((1, hidden), generator=g, device="cuda")
    resid, kv_len = start.clone(), torch.tensor([300], dtype=torch.int32, device="cuda")
    x, x_next = (torch.empty((1, hidden), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    M.moe_rmsnorm_residual(resid, None, x, 1, hidden, 1e-6)
    layer.reserve(1, 1)
    layer.forward(x, resid, x_next, kv_len, table, stream=side)
    torch.cuda.synchronize()
    want = resid.clone(), x_next.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin()
        with torch.cuda.stream(torch.cuda.Stream()):
            layer.forward(x, resid, x_next, kv_len, table, stream=side)
        graph.capture_end()
    assert layer._captured
    many = torch.zeros((300, hidden), device="cuda")
    x_many = torch.zeros((300, hidden), dtype=torch.bfloat16, device="cuda")
    layer.forward(x_many, many, torch.empty_like(x_many), kv_len, table)
    held = [torch.full((300, hidden), 7.0, device="cuda") for _ in range(64)]
    layer.cache.k.zero_(), layer.cache.v.zero_()
    resid.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(resid, want[0]) and torch.equal(x_next, want[1])
    assert all((h == 7.0).all() for h in held)


def test_a_graph_keeps_the_moe_workspace_of_its_calls(M):
    """The MoE half called by itself with more tokens: graphs of it, and of the decoder layer, keep what they use."""
    from test_gpu_decoder_layer import build

    layer = build(M, seed=6)
    hidden = layer.moe.dims.hidden
    g = torch.Generator(device="cuda").manual_seed(4)
    layer.cache.grow(0, 100)
    table, kv_len = layer.cache.table([0]), torch.tensor([100], dtype=torch.int32, device="cuda")
    start = torch.randn((1, hidden), generator=g, device="cuda")
    resid = start.clone()
    x, x_next, y = (torch.empty((1, hidden), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    M.moe_rmsnorm_residual(resid, None, x, 1, hidden, 1e-6)

    def step():
        layer.forward(x, resid, x_next, kv_len, table)
        layer.moe.forward(x, out=y)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (resid, x_next, y)]
    assert not binding.stream_captured() and not layer.moe._captured
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert binding.stream_captured() and binding.stream_captured(torch.cuda.current_stream())
        step()
    assert layer.moe._captured
    many = torch.zeros((500, hidden), dtype=torch.bfloat16, device="cuda")
    size = layer.moe.workspace.numel()
    layer.moe.forward(many)
    assert layer.moe.workspace.numel() > size
    held = [torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(32)]
    for _ in range(2):
        resid.copy_(start)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((resid, x_next, y), want):
            assert torch.equal(a, b)
        assert all((h == 0xff).all() for h in held)
    layer.check_status()

