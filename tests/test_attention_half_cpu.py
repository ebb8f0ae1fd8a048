"""The attention half on the CPU: index arithmetic against brute force, and the refusals of its entry points (every
one before the device is touched; the pointers here are never dereferenced)."""
import ctypes
import math
import os
import subprocess

import pytest

import __graft_entry__
from bit_block_quantized_moe_b200 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, ALIGN, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return B.lib()


def test_index_arithmetic_against_brute_force(tmp_path):
    exe = str(tmp_path / "check")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I",
                           os.path.join(ROOT, "bit_block_quantized_moe_b200", "csrc"),
                           os.path.join(ROOT, "tests", "attn_index_check.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


def test_linear_refusals(lib):
    ws = B.moe_linear_workspace_bytes(64, 256, 128)
    assert ws > 256

    def call(x=0x100000, ld=256, w=0x200000, bias=0x300000, act=0, resid=None, out=0x400000, T=64, K=256, N=128,
             wsp=0x800000, wsb=ws):
        return lib.moe_linear(x, ld, w, bias, act, resid, out, T, K, N, wsp, wsb, None)

    assert call(T=0) == 0
    for bad in (dict(T=-1), dict(T=(1 << 30) + 1), dict(K=0), dict(K=4), dict(K=250), dict(K=65544), dict(N=0), dict(N=262145), dict(act=3),
                dict(act=-1), dict(x=None), dict(w=None), dict(out=None), dict(wsp=None), dict(ld=248), dict(ld=260),
                dict(out=0x100000 + 4096), dict(out=0x200000), dict(out=0x300000 - 16),
                dict(resid=0x400000 + 16), dict(resid=0x400000 - 64)):
        assert call(**bad) == ARG, bad
    for bad in (dict(x=0x100008), dict(w=0x200002), dict(bias=0x300004), dict(out=0x400008), dict(wsp=0x800010 - 8),
                dict(resid=0x500004)):
        assert call(**bad) == ALIGN, bad
    assert call(wsb=ws - 1) == WORKSPACE
    assert B.moe_linear_workspace_bytes(-1, 256, 128) == 0
    assert B.moe_linear_workspace_bytes(8, 12, 128) == 0


def test_linear_workspace_never_shrinks():
    for K, N in ((8, 1), (2048, 2560), (65536, 262144)):
        prev = 0
        for T in (0, 1, 8, 16, 17, 64, 100, 1000, 32768):
            need = B.moe_linear_workspace_bytes(T, K, N)
            assert need >= prev
            prev = need


BAD_DIMS = [(16, 3, 128, 64), (16, 0, 128, 64), (0, 1, 128, 64), (16, 2, 96, 64), (16, 2, 256, 64), (16, 2, 128, 48),
            (16, 2, 128, 8), (16, 2, 128, 256), (1040, 16, 64, 64), (256, 1, 64, 16)]


@pytest.mark.parametrize("dims", BAD_DIMS)
def test_bad_attention_dims(lib, dims):
    d = B.moe_attn_dims(*dims)
    assert B.moe_attn_workspace_bytes(d, 4, 64) == 0
    cache, batch = B.moe_kv_cache(0x1000, 0x2000, 1), B.moe_kv_batch(1, 1, None, 0x3000, 0x4000)
    assert lib.moe_attn_forward(ctypes.byref(d), 0x10000, 1 << 20, ctypes.byref(cache), ctypes.byref(batch), 1, 1.0, 0,
                                0, 0x20000, 0x30000, 1 << 40, None) == ARG


def test_attention_refusals(lib):
    d = B.moe_attn_dims(4, 2, 64, 16)
    ws = B.moe_attn_workspace_bytes(d, 3, 6)
    assert ws > 256 and B.moe_attn_workspace_bytes(d, 0, 6) == 0 and B.moe_attn_workspace_bytes(d, 3, -1) == 0

    def parts(k=0x1000000, v=0x2000000, pages=8, seqs=3, max_pages=5, start=None, lens=0x3000000, table=0x4000000):
        return B.moe_kv_cache(k, v, pages), B.moe_kv_batch(seqs, max_pages, start, lens, table)

    def attn(q=0x100000, ld=256, T=6, scale=0.125, window=0, sinks=0, out=0x200000, wsp=0x300000, wsb=ws, **kw):
        c, b = parts(**kw)
        return lib.moe_attn_forward(ctypes.byref(d), q, ld, ctypes.byref(c), ctypes.byref(b), T, scale, window, sinks,
                                    out, wsp, wsb, None)

    def norm(qkv=0x100000, ld=512, T=6, eps=1e-6, rope=None, out=0x200000, wsp=0x300000, wsb=ws, gq=None, gk=None,
             **kw):
        c, b = parts(**kw)
        return lib.moe_qk_norm_rope(ctypes.byref(d), qkv, ld, gq, gk, eps, None if rope is None else ctypes.byref(rope),
                                    ctypes.byref(c), ctypes.byref(b), T, out, wsp, wsb, None)

    both = (dict(T=-1), dict(T=7), dict(out=None), dict(wsp=None), dict(k=None), dict(v=None), dict(pages=0),
            dict(pages=1 << 27), dict(seqs=0), dict(seqs=65537), dict(max_pages=0), dict(max_pages=(1 << 26) + 1),
            dict(lens=None), dict(table=None), dict(ld=248), dict(ld=514), dict(out=0x100000 + 64),
            dict(out=0x1000000), dict(out=0x2000000 + 4096))
    for fn in (attn, norm):
        assert fn(T=0) == 0
        for bad in both:
            assert fn(**bad) == ARG, (fn.__name__, bad)
        for bad in (dict(out=0x200008), dict(wsp=0x300008), dict(k=0x1000008), dict(v=0x2000002)):
            assert fn(**bad) == ALIGN, (fn.__name__, bad)
        assert fn(wsb=ws - 1) == WORKSPACE
    for bad in (dict(q=None), dict(window=-1), dict(sinks=-1), dict(scale=math.nan), dict(scale=math.inf)):
        assert attn(**bad) == ARG, bad
    assert attn(q=0x100008) == ALIGN
    rope = B.moe_rope_init(1e6, 64)
    wide = B.moe_rope_init(1e6, 128)
    broken = B.moe_rope_init(1e6, 64)
    broken.rotary_dim = 24
    for bad in (dict(qkv=None), dict(eps=-1.0), dict(eps=math.nan), dict(rope=wide), dict(rope=broken),
                dict(k=0x100000 - 4096), dict(v=0x1000000 + 64)):
        assert norm(**bad) == ARG, bad
    assert norm(qkv=0x100004, rope=rope) == ALIGN
    assert norm(gq=0x500004) == ALIGN and norm(gk=0x500008) == ALIGN


def test_rope_table():
    with pytest.raises(B.MoeError):
        B.moe_rope_init(0.5, 64)
    for bad in (0, 8, 24, 144, -16):
        with pytest.raises(B.MoeError):
            B.moe_rope_init(1e4, bad)
    for theta in (1.0, 1e4, 1e6, 1e7):
        for r in (16, 32, 64, 128):
            rope = B.moe_rope_init(theta, r)
            for i in range(r // 2):
                # 2^-64 of a turn for the last place of the table, 2^-52 relative for this check's doubles
                want = theta ** (-2.0 * i / r) / (2 * math.pi) * 2.0 ** 64
                assert abs(rope.turn[i] - want) <= 1 + want * 2.0 ** -50
            assert all(rope.turn[i] == 0 for i in range(r // 2, 64))


def test_paged_cache_bookkeeping(lib):
    import torch

    from bit_block_quantized_moe_b200 import PagedKvCache

    c = PagedKvCache(6, 4, 2, 64, 16, device="cpu")
    assert c.k.shape == c.v.shape == (6, 2, 16, 64)
    c.grow(3, 17)
    c.grow(9, 1)
    assert len(c.pages[3]) == 2 and len(c.pages[9]) == 1
    first = list(c.pages[3])
    c.grow(3, 32)
    assert c.pages[3] == first
    c.grow(3, 33)
    assert c.pages[3][:2] == first and len(set(c.pages[3] + c.pages[9])) == 4
    t = c.table([9, 3, 5])
    assert t.dtype == torch.int32 and t.shape == (3, 3)
    assert t[0, 1:].tolist() == [-1, -1] and t[1].tolist() == c.pages[3] and t[2].tolist() == [-1, -1, -1]
    with pytest.raises(RuntimeError):
        c.grow(5, 100)
    c.release(3)
    c.release(77)
    c.grow(5, 80)
    assert sorted(c.pages[5] + c.pages[9]) == list(range(6))
    with pytest.raises(ValueError):
        PagedKvCache(6, 4, 3, 64, 16, device="cpu")
