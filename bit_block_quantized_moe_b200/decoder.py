"""The other half of a layer: PagedKvCache and Q2DecoderLayer, which runs attention and then its Q2MoeLayer."""
from __future__ import annotations

import torch

from . import binding as B
from .layer import Q2MoeLayer, stream_made_current


class PagedKvCache:
    """The keys and values of one layer in pages, and the page table of each sequence.

    ``k`` and ``v`` are [n_pages, n_kv_heads, page_size, head_dim] bf16.  ``grow`` gives sequences pages from a free
    list on the host; a program with an allocator of its own passes its own tables to ``Q2DecoderLayer.forward``.
    """

    def __init__(self, n_pages: int, n_heads: int, n_kv_heads: int, head_dim: int, page_size: int = 64, device="cuda"):
        self.dims = B.moe_attn_dims(n_heads, n_kv_heads, head_dim, page_size)
        if B.moe_attn_workspace_bytes(self.dims, 1, 1) == 0:
            raise ValueError("unsupported attention dimensions")
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.v = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.free = list(range(n_pages - 1, -1, -1))
        self.pages: dict[int, list[int]] = {}

    def grow(self, seq: int, length: int):
        """Gives sequence `seq` pages for `length` tokens (its earlier ones stay)."""
        have = self.pages.setdefault(seq, [])
        need = -(-length // self.dims.page_size) - len(have)
        if need > len(self.free):
            raise RuntimeError(f"no pages left: sequence {seq} needs {need}, {len(self.free)} are free")
        for _ in range(need):
            have.append(self.free.pop())

    def release(self, seq: int):
        self.free.extend(self.pages.pop(seq, []))

    def table(self, seqs) -> torch.Tensor:
        """[len(seqs), max_pages] int32 on the cache's device, -1 behind each sequence's last page."""
        rows = [self.pages.get(s, []) for s in seqs]
        width = max([1] + [len(r) for r in rows])
        host = torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32)
        return host.to(self.k.device)


class Q2DecoderLayer:
    """One layer of a stack: x += Attention(RMSNorm(x)), then x += MoE(RMSNorm(x)).

    w_qkv [(n_heads + 2 n_kv_heads) * head_dim, hidden] and w_out [hidden, n_heads * head_dim] bf16, b_qkv fp32 or
    None, q_gain and k_gain [head_dim] fp32 or None; moe: the layer's Q2MoeLayer.  Gains of the layer norms are folded
    into w_qkv and the router, as moe_rmsnorm_residual has unit gain.  window 0: all earlier tokens.
    """

    def __init__(self, moe: Q2MoeLayer, cache: PagedKvCache, w_qkv, w_out, b_qkv=None, q_gain=None, k_gain=None,
                 rope_theta: float = 1e6, rotary_dim: int | None = None, window: int = 0, n_sinks: int = 0,
                 eps: float = 1e-6):
        d, hidden = cache.dims, moe.dims.hidden
        width = (d.n_heads + 2 * d.n_kv_heads) * d.head_dim
        if tuple(w_qkv.shape) != (width, hidden) or tuple(w_out.shape) != (hidden, d.n_heads * d.head_dim):
            raise ValueError(f"w_qkv is [{width}, {hidden}], w_out [{hidden}, {d.n_heads * d.head_dim}]")
        self.moe, self.cache, self.eps = moe, cache, eps
        bf16 = dict(device=moe.device, dtype=torch.bfloat16)
        self.w_qkv, self.w_out = w_qkv.to(**bf16).contiguous(), w_out.to(**bf16).contiguous()
        f32 = lambda t: None if t is None else t.to(moe.device, torch.float32).contiguous()  # noqa: E731
        self.b_qkv, self.q_gain, self.k_gain = f32(b_qkv), f32(q_gain), f32(k_gain)
        self.rope = B.moe_rope_init(rope_theta, d.head_dim if rotary_dim is None else rotary_dim)
        self.window, self.n_sinks = window, n_sinks
        self._reserved = (-1, -1)
        self._captured, self._kept = False, []

    def reserve(self, T: int, n_seqs: int):
        """Activations and workspace for calls of up to T tokens and n_seqs sequences, as for Q2MoeLayer shared by all
        calls of this layer: two that can run at the same time need a layer each.  Ready for a call on any stream when
        this returns."""
        old = (*self._buffers(), self.moe.workspace)
        if self._grow(T, n_seqs):
            torch.cuda.synchronize(self.moe.device)  # they are filled, and calls on any stream are done with the old
        del old

    def _buffers(self):
        return (self._qkv, self._q, self._o, self._mid, self._ws) if self._reserved[0] >= 0 else ()

    def _grow(self, T: int, n_seqs: int) -> bool:
        """Makes larger buffers, filled in the order of the current stream."""
        if T <= self._reserved[0] and n_seqs <= self._reserved[1]:
            return False
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("reserve the largest call before capturing one")
        old = self._buffers()
        if self._captured:  # a graph that still reads and writes the smaller buffers
            self._kept.append(old)
        T, n_seqs = max(T, self._reserved[0]), max(n_seqs, self._reserved[1])
        d, hidden, dev = self.cache.dims, self.moe.dims.hidden, self.moe.device
        for t in old:
            # a call on this stream follows the calls before it, with which it shared these; made on another stream,
            # they could be reused there while those still run
            t.record_stream(torch.cuda.current_stream(dev))
        rows = lambda n: torch.empty((T, n), dtype=torch.bfloat16, device=dev)  # noqa: E731
        self._qkv, self._q, self._o = rows(self.w_qkv.shape[0]), rows(self.w_out.shape[1]), rows(self.w_out.shape[1])
        self._mid = rows(hidden)
        self._ws = torch.zeros(max(B.moe_attn_workspace_bytes(d, n_seqs, T),
                                   B.moe_linear_workspace_bytes(T, hidden, self.w_qkv.shape[0]),
                                   B.moe_linear_workspace_bytes(T, self.w_out.shape[1], hidden)),
                               dtype=torch.uint8, device=dev)
        self.moe._grow(T)
        self._reserved = (T, n_seqs)
        return True

    def _prepare(self, T: int, n_seqs: int, stream):
        """A call is about to run on `stream`."""
        if T > self._reserved[0] or n_seqs > self._reserved[1]:
            with stream_made_current(stream, self.moe.device):
                self._grow(T, n_seqs)
        self._captured = self._captured or B.stream_captured(stream)

    def forward(self, x_norm, resid, x_norm_out, kv_len, page_table, q_start=None, stream=None):
        """x_norm [T, hidden] bf16: the RMSNorm of resid [T, hidden] fp32 (moe_rmsnorm_residual, or the layer before);
        resid is updated in place and x_norm_out receives the next layer's input.  The new tokens are already counted
        in kv_len [n_seqs]; page_table and q_start as in moe_attn_forward.  Every row belongs to a sequence: padding
        is one with kv_len 0, whose rows attention leaves as they are."""
        T = x_norm.shape[0]
        if T == 0:
            return x_norm_out
        self._prepare(T, kv_len.shape[0], stream)
        c, ws = self.cache, self._ws
        x = x_norm if x_norm.dtype == torch.bfloat16 else x_norm.view(torch.bfloat16)
        qkv, q, o, mid = self._qkv[:T], self._q[:T], self._o[:T], self._mid[:T]
        B.moe_linear(x, self.w_qkv, qkv, ws, bias=self.b_qkv, stream=stream)
        B.moe_qk_norm_rope(c.dims, qkv, q, c.k, c.v, kv_len, page_table, ws, rope=self.rope, q_start=q_start,
                           q_gain=self.q_gain, k_gain=self.k_gain, eps=self.eps, stream=stream)
        B.moe_attn_forward(c.dims, q, o, c.k, c.v, kv_len, page_table, ws, q_start=q_start, window=self.window,
                           n_sinks=self.n_sinks, stream=stream)
        B.moe_linear(o, self.w_out, resid, ws, resid=resid, stream=stream)
        B.moe_rmsnorm_residual(resid, None, mid, T, self.moe.dims.hidden, self.eps, stream)
        return self.moe.forward_residual(mid, resid, x_norm_out, self.eps, stream=stream)

    def check_status(self, stream=None):
        B.moe_check_status(self._ws, stream)
        self.moe.check_status(stream)
