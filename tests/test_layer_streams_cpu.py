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
            stream = kw["stream"] if "stream" in kw else a[-1]
            self.log.append((name, self.current if stream is None else getattr(stream, "cuda_stream", stream),
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
    monkeypatch.setattr(B, "_stream", lambda s, dev=None: c.current if s is None else getattr(s, "cuda_stream", s))
    monkeypatch.setattr(B, "stream_captured", lambda s=None: bool(c.capturing) and B._stream(s) == c.capturing)
    monkeypatch.setattr(B, "moe_workspace_bytes", lambda dims, T: 16 * (T + 1))
    for name in ("moe_layer_forward", "moe_layer_forward_host", "moe_layer_forward_residual", "moe_experts_forward",
                 "moe_route"):
        monkeypatch.setattr(B, name, c.call(name))
    return c


def moe_layer():
    layer = object.__new__(Q2MoeLayer)
    layer.__dict__.update(dims=B.moe_dims(64, 32, 4, 2), device=torch.device("cpu"), router_w=None, router_b=None,
                          experts=None, shared=None, workspace=None, _ws_T=-1, _captured=False, _kept=[])
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


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("own", [False, True])
def test_moe_graphs_keep_the_workspace_of_their_call(cuda, call, own):
    """A larger call, whoever makes it, takes a workspace of its own when a graph uses the smaller one."""
    layer, stream = moe_layer(), Stream(0x20) if own else None
    x, many = (torch.ones((T, 64), dtype=torch.bfloat16) for T in (3, 9))
    CALLS[call](layer, x, stream)
    CALLS[call](layer, many, stream)
    assert layer._kept == []  # no graph: nothing to keep
    cuda.capturing = 0x20 if own else MAIN
    CALLS[call](layer, x, stream)
    cuda.capturing = False
    used = layer.workspace
    layer.reserve(20)
    assert len(layer._kept) == 1 and layer._kept[0] is used
    CALLS[call](layer, torch.ones((30, 64), dtype=torch.bfloat16), None)
    assert layer.workspace.numel() == 16 * 31


def test_streams_given_as_handles(cuda):
    from bit_block_quantized_moe_b200.layer import stream_made_current

    for given, want in ((None, MAIN), (0, "default"), (1, "default"), (0x40, 0x40), (Stream(0x50), 0x50)):
        with stream_made_current(given, torch.device("cpu")):
            assert cuda.current == want
    assert cuda.current == MAIN


# ---- the decoder layer ---------------------------------------------------------------------------------------------
PARTS = ("moe_linear", "moe_qk_norm_rope", "moe_attn_forward", "moe_linear", "moe_rmsnorm_residual",
         "moe_layer_forward_residual")
BUFFERS = ("_qkv", "_q", "_o", "_mid", "_ws")


@pytest.fixture
def decoder(cuda, monkeypatch):
    from bit_block_quantized_moe_b200.decoder import Q2DecoderLayer

    for name in set(PARTS):
        monkeypatch.setattr(B, name, cuda.call(name))
    monkeypatch.setattr(B, "moe_attn_workspace_bytes", lambda dims, n_seqs, T: 64 * n_seqs + T)
    monkeypatch.setattr(B, "moe_linear_workspace_bytes", lambda T, K, N: 64)
    layer = object.__new__(Q2DecoderLayer)

    class Cache:
        dims, k, v = B.moe_attn_dims(2, 1, 64, 16), None, None

    layer.__dict__.update(moe=moe_layer(), cache=Cache, w_qkv=torch.ones(256, 64), w_out=torch.ones(64, 128), b_qkv=None,
                          q_gain=None, k_gain=None, rope=None, window=0, n_sinks=0, eps=1e-6, _reserved=(-1, -1),
                          _captured=False, _kept=[])

    def call(T, stream, n_seqs=1):
        x = torch.ones((T, 64), dtype=torch.bfloat16)
        layer.forward(x, torch.ones(T, 64), x, torch.ones(n_seqs, dtype=torch.int32), None, stream=stream)

    return layer, call


def buffers(layer):
    return [getattr(layer, n) for n in BUFFERS] + [layer.moe.workspace]


def test_decoder_buffers_are_made_on_the_stream_of_the_call_that_needs_them(cuda, decoder):
    layer, call = decoder
    call(3, Stream(0x20))
    first = buffers(layer)
    assert [cuda.made(t) for t in first] == [0x20] * 6 and cuda.current == MAIN
    assert [(e[0], e[1]) for e in cuda.log if e[0] in PARTS] == [(n, 0x20) for n in PARTS]
    call(2, Stream(0x20))
    assert all(a is b for a, b in zip(buffers(layer), first))
    call(5, Stream(0x30))
    second = buffers(layer)
    assert [cuda.made(t) for t in second] == [0x30] * 6
    assert all(("keep", id(t), 0x30) in cuda.log for t in first)
    call(5, 0x40, n_seqs=4)  # a raw handle, and more sequences alone
    third = buffers(layer)
    assert [cuda.made(t) for t in third[:5]] == [0x40] * 5 and third[5] is second[5]
    assert all(("keep", id(t), 0x40) in cuda.log for t in second[:5])
    call(9, None)
    assert [cuda.made(t) for t in buffers(layer)] == [MAIN] * 6
    assert ("synchronize",) not in cuda.log


def test_decoder_reserve_is_complete_when_it_returns(cuda, decoder):
    layer, _ = decoder
    layer.reserve(4, 2)
    assert cuda.log[-1] == ("synchronize",)
    count = len(cuda.log)
    layer.reserve(4, 1)
    assert len(cuda.log) == count
    layer.reserve(4, 3)
    assert cuda.log[-1] == ("synchronize",)


@pytest.mark.parametrize("own", [False, True])
def test_decoder_knows_that_its_stream_is_captured(cuda, decoder, own):
    """The capture is of the stream that the call runs on, be it the current one or not."""
    layer, call = decoder
    stream = Stream(0x20) if own else None
    call(3, stream)
    assert not layer._captured
    cuda.capturing = 0x20 if own else MAIN
    with pytest.raises(RuntimeError, match="reserve"):
        call(4, stream)
    call(3, stream)
    assert layer._captured
    cuda.capturing = False
    first = buffers(layer)
    call(4, stream)
    assert len(layer._kept) == 1 and all(a is b for a, b in zip(layer._kept[0], first))
