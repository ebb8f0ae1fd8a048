"""Python numbers that the C entry points' 32-bit arguments do not hold: refused, or cut to what means the same, never
taken modulo 2^32.  Tensors without memory stand for the device's."""
import pytest
import torch

from bit_block_quantized_moe_b200 import binding as B

WS = torch.zeros(1 << 21, dtype=torch.uint8)


class Library:
    """The library's entry points, which take down their arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(B, "lib", lambda: fake)
    monkeypatch.setattr(B, "_stream", lambda s, dev=None: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1)
    return fake


def bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="meta")


def i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="meta")


def test_linear_sizes(library):
    B.moe_linear(bf16(5, 64), bf16(3, 64), bf16(5, 3), WS)
    assert library.calls[-1][1][7:10] == (5, 64, 3)
    for T, K, N in ((1 << 32, 8, 1), ((1 << 32) + 1, 8, 1), (1, (1 << 32) + 8, 1), (1, 8, (1 << 32) + 1), (1 << 31, 8, 1)):
        count = len(library.calls)
        with pytest.raises(ValueError):
            B.moe_linear(bf16(T, K), bf16(N, K), bf16(T, N), WS)
        assert len(library.calls) == count, (T, K, N)


def attention(dims, **kw):
    k = bf16(7, dims.n_kv_heads, dims.page_size, dims.head_dim)
    B.moe_attn_forward(dims, bf16(4, 4, 64), bf16(4, 4, 64), k, k, i32(2), i32(2, 3), WS, **kw)


def test_attention_windows_and_sinks(library):
    """Positions lie below 2^30, so that any larger window or number of sinks is all tokens."""
    dims = B.moe_attn_dims(4, 2, 64, 16)
    for given, passed in ((0, 0), (5, 5), (1 << 30, 1 << 30), (1 << 31, 1 << 30), (1 << 32, 1 << 30),
                          ((1 << 32) + 5, 1 << 30), (1 << 63, 1 << 30), (-1, -1), (-(1 << 32) + 5, -1)):
        attention(dims, window=given, n_sinks=0)
        assert library.calls[-1][1][7:9] == (passed, 0), given
        attention(dims, window=5, n_sinks=given)
        assert library.calls[-1][1][7:9] == (5, passed), given


def test_batches_and_caches(library):
    dims = B.moe_attn_dims(4, 2, 64, 16)
    k = bf16(1, 2, 16, 64)
    for shape, cache in ((((1 << 32) + 2, 3), k), ((2, (1 << 32) + 3), k), ((2, 3), bf16((1 << 32) + 1, 2, 16, 64))):
        for run in (lambda *a, **kw: B.moe_attn_forward(dims, bf16(4, 4, 64), bf16(4, 4, 64), *a, **kw),
                    lambda *a, **kw: B.moe_qk_norm_rope(dims, bf16(4, 512), bf16(4, 4, 64), *a, **kw)):
            with pytest.raises(ValueError):
                run(cache, cache, i32(shape[0]), i32(*shape), WS)
    assert library.calls == []
    rows = 1 << 32
    with pytest.raises(ValueError):
        B.moe_attn_forward(dims, bf16(rows, 4, 64), bf16(rows, 4, 64), k, k, i32(2), i32(2, 3), WS)
    with pytest.raises(ValueError):
        B.moe_qk_norm_rope(dims, bf16(rows, 512), bf16(rows, 4, 64), k, k, i32(2), i32(2, 3), WS)
    assert library.calls == []
