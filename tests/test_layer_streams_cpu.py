"""On which stream the layers make, fill and give up their buffers, with stand-ins for the device: a buffer that is
filled on one stream and used on another is a race that a GPU run may or may not show."""
import contextlib

import pytest
import torch

from bit_block_quantized_moe_b200 import binding as B
from bit_block_quantized_moe_b200.layer import Q2MoeLayer

MAIN = 0x10  # a torch stream's handle; the others below are a caller's


class Cuda:
    """The current stream, and what happened on which one, in order."""

    def __init__(self, monkeypatch):
        self.current, self.capturing, self.log, self.alive = MAIN, False, [], []
        patch = lambda name, value: monkeypatch.setattr(torch.cuda, name, value)  # noqa: E731
        patch("stream", self.use)
        patch("ExternalStream", lambda handle, device=None: handle)
        patch("default_stream", lambda device=None: "default")
        patch("current_stream", lambda device=None: self.current)
        patch("is_current_stream_capturing", lambda: self.capturing and self.current == self.capturing)
        patch("synchronize", lambda device=None: self.log.append(("synchronize",)))
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.log.append(("keep", id(t), s)))
        for name in ("zeros", "empty"):
            monkeypatch.setattr(torch, name, self.making(name, getattr(torch, name)))

    @contextlib.contextmanager
    def use(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before

    def making(self, name, make):
        def made(*a, **kw):
            t = make(*a, **kw)
            self.alive.append(t)  # no two with one identity
            self.log.append((name, id(t), self.current))
            return t
        return made

    def call(self, name):
        """A stand-in of a call of the library: its stream, and the tensors that it was given."""
        def called(*a, **kw):
            stream = kw.get("stream", next((x for x in reversed(a) if isinstance(x, Stream)), None))
            self.log.append((name, self.current if stream is None else stream.cuda_stream,
                             [id(x) for x in a if isinstance(x, torch.Tensor)]))
        return called

    def made(self, t):
        return next(e[2] for e in self.log if e[0] in ("zeros", "empty") and e[1] == id(t))


class Stream:
    """What a call takes as a stream: something with a handle."""

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def cuda(monkeypatch):
    c = Cuda(monkeypatch)
    monkeypatch.setattr(B, "moe_workspace_bytes", lambda dims, T: 16 * (T + 1))
    for name in ("moe_layer_forward", "moe_layer_forward_host", "moe_layer_forward_residual", "moe_experts_forward",
                 "moe_route"):
        monkeypatch.setattr(B, name, c.call(name))
    return c


def moe_layer():
    layer = object.__new__(Q2MoeLayer)
    layer.__dict__.update(dims=B.moe_dims(64, 32, 4, 2), device=torch.device("cpu"), router_w=None, router_b=None,
                          experts=None, shared=None, workspace=None, _ws_T=-1)
    return layer


CALLS = {"forward": lambda L, x, s: L.forward(x, stream=s), "forward_host": lambda L, x, s: L.forward_host(x, x, stream=s),
         "forward_residual": lambda L, x, s: L.forward_residual(x, x, x, stream=s),
         "experts_forward": lambda L, x, s: L.experts_forward(x, None, None, stream=s),
         "route": lambda L, x, s: L.route(x, stream=s)}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [Stream(0x20), None])
def test_moe_workspace_is_filled_on_the_stream_of_the_call_that_needs_it(cuda, call, stream):
    layer, x = moe_layer(), torch.ones((3, 64), dtype=torch.bfloat16)
    runs_on = MAIN if stream is None else stream.cuda_stream
    CALLS[call](layer, x, stream)
    first = layer.workspace
    assert cuda.made(first) == runs_on and cuda.current == MAIN
    CALLS[call](layer, x[:2], stream)
    assert layer.workspace is first
    # a larger call on another stream: its own fill, and the old memory is not reused before that stream is done
    many = torch.ones((9, 64), dtype=torch.bfloat16)
    CALLS[call](layer, many, Stream(0x30))
    assert layer.workspace is not first and cuda.made(layer.workspace) == 0x30
    assert ("keep", id(first), 0x30) in cuda.log and ("synchronize",) not in cuda.log


def test_moe_reserve_is_complete_when_it_returns(cuda):
    """No call orders what follows it, so that the host waits: for the fill, and for calls that use the old memory."""
    layer = moe_layer()
    layer.reserve(4)
    assert cuda.log[-1] == ("synchronize",)
    count = len(cuda.log)
    layer.reserve(3)
    assert len(cuda.log) == count
    layer.reserve(5)
    assert cuda.log[-1] == ("synchronize",)
    cuda.capturing = MAIN  # not allowed there
    count = cuda.log.count(("synchronize",))
    layer.reserve(6)
    assert cuda.log.count(("synchronize",)) == count and layer.workspace.numel() == 16 * 7


def test_streams_given_as_handles(cuda):
    from bit_block_quantized_moe_b200.layer import stream_made_current

    for given, want in ((None, MAIN), (0, "default"), (1, "default"), (0x40, 0x40), (Stream(0x50), 0x50)):
        with stream_made_current(given, torch.device("cpu")):
            assert cuda.current == want
    assert cuda.current == MAIN
