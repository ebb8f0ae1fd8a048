"""Q2MoeLayer: owns the device buffers of one layer and calls the C ABI."""
from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import binding as B


def stream_made_current(stream, device):
    """Context in which the `stream` argument of a call (None: as it is, a raw handle, or an object that has one) is the
    current stream of `device`, so that buffers made there are filled, and freed, in its order."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        # 0 and 1 are names of the legacy default stream
        stream = torch.cuda.ExternalStream(handle, device) if handle > 1 else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


class Q2MoeLayer:
    """One routed MoE layer: router (fp32), packed routed experts and packed shared expert.

    Buffers live on ``device``; ``forward`` calls ``moe_layer_forward`` once.
    The canonical Q2 bytes are copied to the device, repacked there by
    ``moe_pack_q2`` and released.
    """

    def __init__(self, hidden: int, inter: int, n_experts: int, top_k: int, router_w, router_b, experts_canon,
                 shared_canon, device="cuda", max_tokens: int = 0):
        self.dims = B.moe_dims(hidden, inter, n_experts, top_k)
        self.device = torch.device(device)
        self.router_w = self._f32(router_w)
        self.router_b = None if router_b is None else self._f32(router_b)
        pe = B.moe_packed_expert_bytes(self.dims)
        ce = B.moe_canonical_expert_bytes(self.dims)
        if pe == 0 or ce == 0:
            raise ValueError("unsupported layer dimensions")
        self.experts = torch.empty(n_experts * pe, dtype=torch.uint8, device=self.device)
        self.shared = torch.empty(pe, dtype=torch.uint8, device=self.device)
        self._pack(experts_canon, n_experts, ce, self.experts)
        self._pack(shared_canon, 1, ce, self.shared)
        self.workspace = None
        self._ws_T = -1
        self._captured, self._kept = False, []
        if max_tokens:
            self.reserve(max_tokens)

    def _f32(self, a):
        if isinstance(a, torch.Tensor):
            return a.detach().to(self.device, torch.float32).contiguous()
        return torch.as_tensor(np.ascontiguousarray(a, dtype=np.float32)).to(self.device)

    def _pack(self, canon, n, ce, dst):
        if isinstance(canon, torch.Tensor):
            src = canon.detach().reshape(-1)
            assert src.dtype == torch.uint8
        else:
            src = torch.as_tensor(np.ascontiguousarray(canon, dtype=np.uint8).reshape(-1))
        assert src.numel() == n * ce
        # pack in slices to bound the temporary device copy
        per = max(1, (256 << 20) // ce)
        pe = B.moe_packed_expert_bytes(self.dims)
        for s in range(0, n, per):
            m = min(per, n - s)
            tmp = src[s * ce:(s + m) * ce].to(self.device)
            B.moe_pack_q2(self.dims, tmp, m, dst[s * pe:(s + m) * pe])
        torch.cuda.synchronize(self.device)

    def reserve(self, T: int):
        """Workspace for calls of up to T tokens, ready for a call on any stream when this returns.  (While a stream is
        captured it is filled by the graph.)"""
        old = self.workspace
        if self._grow(T) and not torch.cuda.is_current_stream_capturing():
            torch.cuda.synchronize(self.device)  # the new one is filled, and calls on any stream are done with the old
        del old

    def _grow(self, T: int) -> bool:
        """Makes a larger workspace, filled in the order of the current stream."""
        if T <= self._ws_T:
            return False
        nbytes = B.moe_workspace_bytes(self.dims, T)
        if self._captured:  # a graph that still uses the smaller one
            self._kept.append(self.workspace)
        if self.workspace is not None:
            # A call on this stream replaces the workspace that it shares with the calls before it, which it follows.
            # Made on another stream, it could be reused there while they still run.
            self.workspace.record_stream(torch.cuda.current_stream(self.device))
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self._ws_T = T
        return True

    def _prepare(self, T: int, stream):
        """A call of T tokens is about to run on `stream`."""
        if T > self._ws_T:
            with stream_made_current(stream, self.device):
                self._grow(T)
        self._captured = self._captured or B.stream_captured(stream)

    def forward(self, x, out=None, topk_idx=None, topk_w=None, stream=None):
        """x: [T, hidden] bf16 (torch.bfloat16 or int16 bit patterns) on device."""
        T = x.shape[0]
        self._prepare(T, stream)
        if out is None:
            out = torch.empty_like(x)
        B.moe_layer_forward(self.dims, x, self.router_w, self.router_b, self.experts, self.shared, out, T,
                            self.workspace, topk_idx, topk_w, stream)
        return out

    def forward_host(self, x_host, out_host=None, topk_idx=None, topk_w=None, stream=None):
        """x_host: [T <= 8, hidden] bf16 bit patterns in page-locked host memory; the output goes to out_host
        (page-locked, allocated if None), complete once the stream has passed the call."""
        T = x_host.shape[0]
        self._prepare(T, stream)
        if out_host is None:
            out_host = torch.empty(x_host.shape, dtype=x_host.dtype).pin_memory()
        B.moe_layer_forward_host(self.dims, x_host, self.router_w, self.router_b, self.experts, self.shared, out_host,
                                 T, self.workspace, topk_idx, topk_w, stream)
        return out_host

    def forward_residual(self, x_norm, resid, x_norm_out, eps=1e-6, topk_idx=None, topk_w=None, stream=None):
        """One stacked layer: resid += layer(x_norm); x_norm_out = bf16(RMSNorm(resid))."""
        T = x_norm.shape[0]
        self._prepare(T, stream)
        B.moe_layer_forward_residual(self.dims, x_norm, self.router_w, self.router_b, self.experts, self.shared, resid,
                                     x_norm_out, T, self.workspace, eps, topk_idx, topk_w, stream)
        return x_norm_out

    def experts_forward(self, x, topk_idx, topk_w, out=None, stream=None):
        T = x.shape[0]
        self._prepare(T, stream)
        if out is None:
            out = torch.empty_like(x)
        B.moe_experts_forward(self.dims, x, topk_idx, topk_w, self.experts, self.shared, out, T, self.workspace,
                              stream)
        return out

    def route(self, x, topk_idx=None, topk_w=None, stream=None):
        T = x.shape[0]
        self._prepare(T, stream)
        k = self.dims.top_k
        if topk_idx is None:
            topk_idx = torch.empty((T, k), dtype=torch.int32, device=self.device)
        if topk_w is None:
            topk_w = torch.empty((T, k), dtype=torch.float32, device=self.device)
        B.moe_route(self.dims, x, self.router_w, self.router_b, T, topk_idx, topk_w, self.workspace, stream)
        return topk_idx, topk_w

    def check_status(self, stream=None):
        B.moe_check_status(self.workspace, stream)
