"""Limits of the attention half's entry points beyond those of test_attention_half_cpu (no device is touched)."""
import ctypes

import pytest

import __graft_entry__
from bit_block_quantized_moe_b200 import binding as B

ARG = 1


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return B.lib()


def test_rows_of_a_call(lib):
    """At most 2^30: the kernels step beyond the last row in 32 bits."""
    d = B.moe_attn_dims(1, 1, 64, 16)
    cache, batch = B.moe_kv_cache(1 << 44, 1 << 45, 1), B.moe_kv_batch(1, 1, None, 0x3000, 0x4000)
    most, ws = 1 << 30, 1 << 40
    assert B.moe_attn_workspace_bytes(d, 1, most) > 0
    for T in (most + 1, (1 << 31) - 1):
        assert B.moe_attn_workspace_bytes(d, 1, T) == 0
        assert lib.moe_attn_forward(ctypes.byref(d), 1 << 40, 64, ctypes.byref(cache), ctypes.byref(batch), T, 1.0, 0, 0,
                                    1 << 42, 0x30000, ws, None) == ARG
        assert lib.moe_qk_norm_rope(ctypes.byref(d), 1 << 40, 192, None, None, 1e-6, None, ctypes.byref(cache),
                                    ctypes.byref(batch), T, 1 << 42, 0x30000, ws, None) == ARG
