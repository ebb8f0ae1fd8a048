"""ctypes binding of include/moe_q2.h (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_q2.so")

MOE_OK = 0
_lib = None


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {moe_status_str(code)} (status {code})")
        self.code = code


class moe_dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32)]


class moe_router(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class moe_experts(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p)]


class moe_shared(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p)]


class moe_attn_dims(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class moe_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int32)]


class moe_kv_batch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p)]


class moe_rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("reserved", ctypes.c_int32), ("turn", ctypes.c_uint64 * 64)]


EXPORTED = [
    "moe_canonical_expert_bytes",
    "moe_packed_expert_bytes",
    "moe_pack_q2",
    "moe_workspace_bytes",
    "moe_route",
    "moe_route_noalloc",
    "moe_layer_forward",
    "moe_layer_forward_host",
    "moe_layer_forward_residual",
    "moe_experts_forward",
    "moe_dispatch",
    "moe_rmsnorm_residual",
    "moe_linear_workspace_bytes",
    "moe_linear",
    "moe_rope_init",
    "moe_attn_workspace_bytes",
    "moe_qk_norm_rope",
    "moe_attn_forward",
    "moe_trace_kernel",
    "moe_set_cold_expert_tokens",
    "moe_check_status",
    "moe_status_str",
]


def lib():
    """Load libmoe_q2.so (built by bit_block_quantized_moe_b200.build); fails loudly if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing (run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        D = ctypes.POINTER(moe_dims)
        L.moe_canonical_expert_bytes.restype = sz
        L.moe_canonical_expert_bytes.argtypes = [D]
        L.moe_packed_expert_bytes.restype = sz
        L.moe_packed_expert_bytes.argtypes = [D]
        L.moe_pack_q2.restype = ctypes.c_int
        L.moe_pack_q2.argtypes = [D, P, i32, P, sz, P]
        L.moe_workspace_bytes.restype = sz
        L.moe_workspace_bytes.argtypes = [D, i32]
        L.moe_route.restype = ctypes.c_int
        L.moe_route.argtypes = [D, P, ctypes.POINTER(moe_router), i32, P, P, P, sz, P]
        L.moe_route_noalloc.restype = ctypes.c_int
        L.moe_route_noalloc.argtypes = [D, P, ctypes.POINTER(moe_router), i32, P, P, P]
        L.moe_layer_forward.restype = ctypes.c_int
        L.moe_layer_forward.argtypes = [D, P, ctypes.POINTER(moe_router), ctypes.POINTER(moe_experts),
                                        ctypes.POINTER(moe_shared), P, i32, P, P, P, sz, P]
        L.moe_layer_forward_host.restype = ctypes.c_int
        L.moe_layer_forward_host.argtypes = [D, P, ctypes.POINTER(moe_router), ctypes.POINTER(moe_experts),
                                             ctypes.POINTER(moe_shared), P, i32, P, P, P, sz, P]
        L.moe_layer_forward_residual.restype = ctypes.c_int
        L.moe_layer_forward_residual.argtypes = [D, P, ctypes.POINTER(moe_router), ctypes.POINTER(moe_experts),
                                                 ctypes.POINTER(moe_shared), P, P, ctypes.c_float, i32, P, P, P, sz,
                                                 P]
        L.moe_experts_forward.restype = ctypes.c_int
        L.moe_experts_forward.argtypes = [D, P, P, P, ctypes.POINTER(moe_experts), ctypes.POINTER(moe_shared), P,
                                          i32, P, sz, P]
        L.moe_dispatch.restype = ctypes.c_int
        L.moe_dispatch.argtypes = [D, P, i32, P, P, P, P, P, sz, P]
        L.moe_rmsnorm_residual.restype = ctypes.c_int
        L.moe_rmsnorm_residual.argtypes = [P, P, P, i32, i32, ctypes.c_float, P]
        i64, f32, A = ctypes.c_int64, ctypes.c_float, ctypes.POINTER(moe_attn_dims)
        C, S = ctypes.POINTER(moe_kv_cache), ctypes.POINTER(moe_kv_batch)
        L.moe_linear_workspace_bytes.restype = sz
        L.moe_linear_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_linear.restype = ctypes.c_int
        L.moe_linear.argtypes = [P, i64, P, P, ctypes.c_int, P, P, i32, i32, i32, P, sz, P]
        L.moe_rope_init.restype = ctypes.c_int
        L.moe_rope_init.argtypes = [ctypes.c_double, i32, ctypes.POINTER(moe_rope)]
        L.moe_attn_workspace_bytes.restype = sz
        L.moe_attn_workspace_bytes.argtypes = [A, i32, i32]
        L.moe_qk_norm_rope.restype = ctypes.c_int
        L.moe_qk_norm_rope.argtypes = [A, P, i64, P, P, f32, ctypes.POINTER(moe_rope), C, S, i32, P, P, sz, P]
        L.moe_attn_forward.restype = ctypes.c_int
        L.moe_attn_forward.argtypes = [A, P, i64, C, S, i32, f32, i32, i32, P, P, sz, P]
        # of the CUDA runtime that the library is linked to
        L.cudaStreamIsCapturing.restype = ctypes.c_int
        L.cudaStreamIsCapturing.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
        L.cudaGetLastError.restype = ctypes.c_int
        L.cudaGetLastError.argtypes = []
        L.moe_trace_kernel.restype = ctypes.c_int
        L.moe_trace_kernel.argtypes = [i32, P, P]
        L.moe_set_cold_expert_tokens.restype = ctypes.c_int
        L.moe_set_cold_expert_tokens.argtypes = [i32]
        L.moe_check_status.restype = ctypes.c_int
        L.moe_check_status.argtypes = [P, P]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_status_str.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, dev=None):
    if stream is None:
        # the handle itself: torch.cuda.current_stream() builds an object around it, 5 us against 0.3
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None else dev)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def stream_captured(stream=None) -> bool:
    """Whether work on `stream` (None: the current one) goes into a graph."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    status = ctypes.c_int(0)
    if lib().cudaStreamIsCapturing(_stream(stream), ctypes.byref(status)) != 0:
        lib().cudaGetLastError()  # the legacy stream while another one is captured: the call itself will say so
    return status.value != 0


def _check(code: int, what: str):
    if code != MOE_OK:
        raise MoeError(code, what)


def _dims(d) -> moe_dims:
    if isinstance(d, moe_dims):
        return d
    return moe_dims(int(d[0]), int(d[1]), int(d[2]), int(d[3]))


def moe_status_str(code: int) -> str:
    return lib().moe_status_str(int(code)).decode()


def moe_canonical_expert_bytes(dims) -> int:
    return int(lib().moe_canonical_expert_bytes(ctypes.byref(_dims(dims))))


def moe_packed_expert_bytes(dims) -> int:
    return int(lib().moe_packed_expert_bytes(ctypes.byref(_dims(dims))))


def moe_workspace_bytes(dims, max_T: int) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(_dims(dims)), int(max_T)))


def moe_pack_q2(dims, canonical, n_experts: int, packed, stream=None):
    code = lib().moe_pack_q2(ctypes.byref(_dims(dims)), _ptr(canonical), int(n_experts), _ptr(packed),
                             packed.numel() * packed.element_size(), _stream(stream))
    _check(code, "moe_pack_q2")


def moe_route(dims, x, router_w, router_b, T: int, topk_idx, topk_w, workspace, stream=None):
    r = moe_router(_ptr(router_w), _ptr(router_b))
    code = lib().moe_route(ctypes.byref(_dims(dims)), _ptr(x), ctypes.byref(r), int(T), _ptr(topk_idx),
                           _ptr(topk_w), _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream(stream))
    _check(code, "moe_route")


def moe_route_noalloc(dims, x, router_w, router_b, T: int, topk_idx, topk_w, stream=None):
    """moe_route without a workspace: the library's own static device scratch holds the
    logits, for callers that cannot allocate device memory (see include/moe_q2.h)."""
    r = moe_router(_ptr(router_w), _ptr(router_b))
    code = lib().moe_route_noalloc(ctypes.byref(_dims(dims)), _ptr(x), ctypes.byref(r), int(T), _ptr(topk_idx),
                                   _ptr(topk_w), _stream(stream))
    _check(code, "moe_route_noalloc")


def moe_layer_forward(dims, x, router_w, router_b, experts_packed, shared_packed, out, T: int, workspace,
                      topk_idx_out=None, topk_w_out=None, stream=None):
    r = moe_router(_ptr(router_w), _ptr(router_b))
    ex = moe_experts(_ptr(experts_packed))
    sh = moe_shared(_ptr(shared_packed))
    code = lib().moe_layer_forward(ctypes.byref(_dims(dims)), _ptr(x), ctypes.byref(r), ctypes.byref(ex),
                                   ctypes.byref(sh), _ptr(out), int(T), _ptr(topk_idx_out), _ptr(topk_w_out),
                                   _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(code, "moe_layer_forward")


def moe_layer_forward_host(dims, x_host, router_w, router_b, experts_packed, shared_packed, out_host, T: int,
                           workspace, topk_idx_out=None, topk_w_out=None, stream=None):
    """x_host / out_host: page-locked host tensors (e.g. torch's pin_memory()), T <= 8."""
    r = moe_router(_ptr(router_w), _ptr(router_b))
    ex = moe_experts(_ptr(experts_packed))
    sh = moe_shared(_ptr(shared_packed))
    code = lib().moe_layer_forward_host(ctypes.byref(_dims(dims)), _ptr(x_host), ctypes.byref(r), ctypes.byref(ex),
                                        ctypes.byref(sh), _ptr(out_host), int(T), _ptr(topk_idx_out),
                                        _ptr(topk_w_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream))
    _check(code, "moe_layer_forward_host")


def moe_layer_forward_residual(dims, x_norm_in, router_w, router_b, experts_packed, shared_packed, resid, x_norm_out,
                               T: int, workspace, eps: float = 1e-6, topk_idx_out=None, topk_w_out=None,
                               stream=None):
    r = moe_router(_ptr(router_w), _ptr(router_b))
    ex = moe_experts(_ptr(experts_packed))
    sh = moe_shared(_ptr(shared_packed))
    code = lib().moe_layer_forward_residual(ctypes.byref(_dims(dims)), _ptr(x_norm_in), ctypes.byref(r),
                                            ctypes.byref(ex), ctypes.byref(sh), _ptr(resid), _ptr(x_norm_out),
                                            float(eps), int(T), _ptr(topk_idx_out), _ptr(topk_w_out),
                                            _ptr(workspace), workspace.numel() * workspace.element_size(),
                                            _stream(stream))
    _check(code, "moe_layer_forward_residual")


def moe_experts_forward(dims, x, topk_idx, topk_w, experts_packed, shared_packed, out, T: int, workspace,
                        stream=None):
    ex = moe_experts(_ptr(experts_packed))
    sh = moe_shared(_ptr(shared_packed))
    code = lib().moe_experts_forward(ctypes.byref(_dims(dims)), _ptr(x), _ptr(topk_idx), _ptr(topk_w),
                                     ctypes.byref(ex), ctypes.byref(sh), _ptr(out), int(T), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream))
    _check(code, "moe_experts_forward")


def moe_dispatch(dims, topk_idx, T: int, counts, offsets, perm, inv, workspace, stream=None):
    code = lib().moe_dispatch(ctypes.byref(_dims(dims)), _ptr(topk_idx), int(T), _ptr(counts), _ptr(offsets),
                              _ptr(perm), _ptr(inv), _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream))
    _check(code, "moe_dispatch")


def moe_rmsnorm_residual(resid, y, x_norm, T: int, hidden: int, eps: float = 1e-6, stream=None):
    code = lib().moe_rmsnorm_residual(_ptr(resid), _ptr(y), _ptr(x_norm), int(T), int(hidden), float(eps),
                                      _stream(stream))
    _check(code, "moe_rmsnorm_residual")


MOE_ACT = {"none": 0, "silu": 1, "gelu": 2}


# ctypes takes larger sizes modulo 2^32
_INT32_END = 1 << 31
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_I32, _F32 = torch.int32, torch.float32


def _check_tensors(what, half, others):
    """Every tensor on the current CUDA device (the call launches there), which is returned; `half` in bf16, or its bit
    patterns in 16-bit integers."""
    dev = torch._C._cuda_getDevice()  # torch.cuda.current_device() asks for the initialisation too, 0.2 us
    for t in half:
        if t.get_device() != dev or t.dtype not in _BF16:
            raise ValueError(f"{what}: activations, weights and caches are bf16, on the current CUDA device")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{what}: every tensor belongs on the current CUDA device")
    return dev


def moe_linear_workspace_bytes(max_T: int, K: int, N: int) -> int:
    return int(lib().moe_linear_workspace_bytes(int(max_T), int(K), int(N)))


def moe_linear(x, w, out, workspace, bias=None, act="none", resid=None, stream=None):
    """out = act(x w^T + bias) in bf16, or resid + that in fp32 (out may be resid).  x [T, K] bf16 (rows may be
    strided), w [N, K] bf16, bias [N] fp32, resid and out [T, N]."""
    dev = _check_tensors("moe_linear", (x, w), (out, workspace, bias, resid))
    T, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K or out.shape != (T, N) or (bias is not None and (bias.numel() != N or bias.dtype != _F32)) or (
            resid is not None and (resid.shape != (T, N) or resid.dtype != _F32)) or max(T, K, N) >= _INT32_END:
        raise ValueError("moe_linear: shapes or types do not match, or are too large")
    if act not in MOE_ACT or (out.dtype != _F32 if resid is not None else out.dtype not in _BF16):
        raise ValueError("moe_linear: out is bf16, or fp32 with a residual; act is none, silu or gelu")
    if x.stride(1) != 1 or not (w.is_contiguous() and out.is_contiguous() and (bias is None or bias.is_contiguous())
                                and (resid is None or resid.is_contiguous())):
        raise ValueError("moe_linear: only the rows of x may be strided")
    code = lib().moe_linear(x.data_ptr(), x.stride(0) if T > 1 else K, w.data_ptr(), _ptr(bias), MOE_ACT[act],
                            _ptr(resid), out.data_ptr(), T, K, N, workspace.data_ptr(), workspace.nbytes,
                            _stream(stream, dev))
    _check(code, "moe_linear")


def moe_rope_init(theta: float, rotary_dim: int) -> moe_rope:
    rope = moe_rope()
    _check(lib().moe_rope_init(float(theta), int(rotary_dim), ctypes.byref(rope)), "moe_rope_init")
    return rope


def moe_attn_workspace_bytes(dims: moe_attn_dims, n_seqs: int, max_T: int) -> int:
    return int(lib().moe_attn_workspace_bytes(ctypes.byref(dims), int(n_seqs), int(max_T)))


def _cache_and_batch(what, dims, k_cache, v_cache, kv_len, page_table, q_start):
    shape = k_cache.shape
    if shape[1:] != (dims.n_kv_heads, dims.page_size, dims.head_dim) or v_cache.shape != shape or not (
            k_cache.is_contiguous() and v_cache.is_contiguous()) or shape[0] >= _INT32_END:
        raise ValueError(f"{what}: k and v are contiguous [n_pages, n_kv_heads, page_size, head_dim]")
    n, pages = page_table.shape
    if kv_len.numel() != n or page_table.dtype != _I32 or kv_len.dtype != _I32 or not (
            page_table.is_contiguous() and kv_len.is_contiguous()) or (q_start is not None and (
                q_start.numel() != n + 1 or q_start.dtype != _I32 or not q_start.is_contiguous())) or (
                    max(n, pages) >= _INT32_END):
        raise ValueError(f"{what}: kv_len [n_seqs], page_table [n_seqs, max_pages], q_start [n_seqs + 1], contiguous "
                         "int32")
    return (moe_kv_cache(k_cache.data_ptr(), v_cache.data_ptr(), shape[0]),
            moe_kv_batch(n, pages, _ptr(q_start), kv_len.data_ptr(), page_table.data_ptr()))


def _token_rows(what, t, heads, dim):
    """Elements between neighbouring tokens of t, [T, heads, dim] or [T, heads * dim]."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        ok = shape[1] == heads and shape[2] == dim and stride[2] == 1 and (heads == 1 or stride[1] == dim)
    else:
        ok = len(shape) == 2 and shape[1] == heads * dim and stride[1] == 1
    if not ok or shape[0] >= _INT32_END:
        raise ValueError(f"{what} [T, {heads}, {dim}], every token contiguous")
    return stride[0] if shape[0] > 1 else heads * dim


def moe_qk_norm_rope(dims, qkv, q_out, k_cache, v_cache, kv_len, page_table, workspace, rope=None, q_start=None,
                     q_gain=None, k_gain=None, eps=1e-6, stream=None):
    """Per-head norms and rotation of qkv [T, (n_heads + 2 n_kv_heads) * head_dim]; queries to q_out [T, n_heads,
    head_dim], keys and values to their pages."""
    what = "moe_qk_norm_rope"
    dev = _check_tensors(what, (qkv, q_out, k_cache, v_cache), (kv_len, page_table, workspace, q_start, q_gain, k_gain))
    cache, batch = _cache_and_batch(what, dims, k_cache, v_cache, kv_len, page_table, q_start)
    ld = _token_rows("moe_qk_norm_rope: qkv", qkv, dims.n_heads + 2 * dims.n_kv_heads, dims.head_dim)
    T = qkv.shape[0]
    if q_out.shape[0] != T or q_out.numel() != T * dims.n_heads * dims.head_dim or not q_out.is_contiguous():
        raise ValueError("moe_qk_norm_rope: q_out is contiguous [T, n_heads, head_dim]")
    for gain in (q_gain, k_gain):
        if gain is not None and (gain.dtype != _F32 or gain.numel() != dims.head_dim
                                 or not gain.is_contiguous()):
            raise ValueError("moe_qk_norm_rope: gains are [head_dim] fp32")
    code = lib().moe_qk_norm_rope(ctypes.byref(dims), qkv.data_ptr(), ld, _ptr(q_gain), _ptr(k_gain), eps,
                                  None if rope is None else ctypes.byref(rope), ctypes.byref(cache),
                                  ctypes.byref(batch), T, q_out.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                  _stream(stream, dev))
    _check(code, what)


def _tokens(n):
    """A window or a number of sinks as the library takes it: 2^30 and more are all tokens, below 0 is refused there."""
    return n if 0 <= n <= 1 << 30 else -1 if n < 0 else 1 << 30


def moe_attn_forward(dims, q, out, k_cache, v_cache, kv_len, page_table, workspace, q_start=None, scale=None, window=0,
                     n_sinks=0, stream=None):
    """Attention of q [T, n_heads, head_dim] (tokens may be strided) over the paged cache; scale defaults to
    head_dim ** -0.5."""
    what = "moe_attn_forward"
    dev = _check_tensors(what, (q, out, k_cache, v_cache), (kv_len, page_table, workspace, q_start))
    cache, batch = _cache_and_batch(what, dims, k_cache, v_cache, kv_len, page_table, q_start)
    ld = _token_rows("moe_attn_forward: q", q, dims.n_heads, dims.head_dim)
    T = q.shape[0]
    if out.shape[0] != T or out.numel() != T * dims.n_heads * dims.head_dim or not out.is_contiguous():
        raise ValueError("moe_attn_forward: out is contiguous [T, n_heads, head_dim]")
    code = lib().moe_attn_forward(ctypes.byref(dims), q.data_ptr(), ld, ctypes.byref(cache), ctypes.byref(batch), T,
                                  dims.head_dim ** -0.5 if scale is None else scale, _tokens(window), _tokens(n_sinks),
                                  out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _stream(stream, dev))
    _check(code, what)


MOE_KERNEL = {"router_logits": 0, "topk": 1, "dispatch_bits": 2, "dispatch_scan": 3, "dispatch_place": 4,
              "gate_up": 5, "down": 6, "combine": 7, "decode_fused": 8,
              "gather": 9, "linear": 10, "qk_norm": 11, "attn": 12}


def moe_trace_kernel(kernel_id: int, before=None, after=None):
    """Record torch.cuda.Event `before`/`after` (created with external=True) around kernel `kernel_id`."""
    b = None if before is None else before.cuda_event
    a = None if after is None else after.cuda_event
    _check(lib().moe_trace_kernel(int(kernel_id), b, a), "moe_trace_kernel")


def moe_set_cold_expert_tokens(max_tokens: int):
    """Per host thread: in a prefill chunk, experts with at most max_tokens tokens run on the register-dequant
    kernels (0, the default: every expert on the tcgen05 kernels)."""
    _check(lib().moe_set_cold_expert_tokens(int(max_tokens)), "moe_set_cold_expert_tokens")


def moe_check_status(workspace, stream=None):
    code = lib().moe_check_status(_ptr(workspace), _stream(stream))
    _check(code, "moe_check_status")
