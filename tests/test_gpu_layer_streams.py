"""Layers called on a stream of their own while the current stream is busy: the same results as on the current stream,
for a first call, for a larger one behind it, and for one with a raw handle."""
import numpy as np
import pytest
import torch

from gen import CONFIGS, make_layer, make_x

pytestmark = pytest.mark.gpu

BUSY = 50_000_000  # clock cycles: 25 ms, far more than all calls here together


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
