"""Exact fused attention forward on GB300 (sm_103a): a thin ctypes binding over libfa.so.

The binding only marshals arguments: every step of the computation runs in the CUDA
kernels of ``libfa.so`` (source in ``csrc/``, C ABI in ``include/fa_fwd.h`` and
``include/fa_decoder.h``). There is
no CPU or PyTorch fallback: importing this package fails loudly when the library has
not been built (``python -c "import __graft_entry__ as g; g.build()"``).

Function names follow the C ABI:
    fa_fwd(Q, K, V, O, L, B, H, Nq, Nk, d, scale, causal, dtype, stream) -> status
plus a tensor-level convenience ``attention(q, k, v, causal, scale)`` -> (O, L), and for the
operators next to it in a decoder block ``qk_norm_rope``, ``qk_norm_rope_backward``,
``paged_append`` and ``attention_paged``, for a cache held in 8 bits ``paged_append_fp8`` and
``attention_paged_fp8``, for eviction from either ``paged_key_weights`` and ``paged_evict``.
"""
from __future__ import annotations

import ctypes
import math
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfa.so")
# The same library built with FA_DEBUG: every stream-K workspace access and TMA tile
# coordinate of the forward kernel is range-checked on the device, and a violation is
# recorded as FA_ERR_BOUNDS. Tests load it with load_library; FA_LIBRARY=debug in the
# environment makes it the library this module binds.
DEBUG_LIB_PATH = os.path.join(PKG, "libfa_debug.so")
# The native tensor-level calls of the decoder-block operators (csrc/fa_torch.cpp).
TORCH_CALLS_PATH = os.path.join(PKG, "_fa_torch.so")

FA_F16 = 0
FA_BF16 = 1

STATUS = {
    0: "FA_OK", -1: "FA_ERR_NULL", -2: "FA_ERR_HEAD_DIM", -3: "FA_ERR_SHAPE",
    -4: "FA_ERR_EMPTY_KEYS", -5: "FA_ERR_SCALE", -6: "FA_ERR_ALIGN", -7: "FA_ERR_DTYPE",
    -8: "FA_ERR_CUDA", -9: "FA_ERR_TENSOR_MAP", -10: "FA_ERR_DEVICE", -11: "FA_ERR_TIMEOUT",
    -12: "FA_ERR_WORKSPACE", -13: "FA_ERR_SCRATCH_LIMIT", -14: "FA_ERR_DROPOUT",
    -15: "FA_ERR_RANGE", -16: "FA_ERR_BOUNDS",
}
FA_WAIT_LIMIT_DEFAULT_US = 2_000_000
FA_WAIT_LIMIT_MIN_US = 100
FA_WAIT_LIMIT_MAX_US = 3_600_000_000
FA_NOALLOC_SCRATCH_BYTES = 48 << 20
globals().update({v: k for k, v in STATUS.items()})


class fa_heads(ctypes.Structure):
    """Rows of d elements by (batch, token, head); strides in elements (see fa_decoder.h)."""
    _fields_ = [("ptr", ctypes.c_void_p), ("batch_stride", ctypes.c_longlong),
                ("token_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong), ("H", ctypes.c_int)]


class fa_paged_kv(ctypes.Structure):
    """A paged cache of keys and values (see fa_decoder.h)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("token_stride", ctypes.c_longlong),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int)]


class fa_rope(ctypes.Structure):
    """A rotation table (see fa_decoder.h)."""
    _fields_ = [("table", ctypes.c_void_p), ("length", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int)]


class FAError(RuntimeError):
    def __init__(self, code: int, what: str = "fa_fwd"):
        self.code = code
        super().__init__(f"{what} failed: {STATUS.get(code, code)} ({strerror(code)})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Open one build of the library (release or FA_DEBUG) with its C signatures declared."""
    if not os.path.exists(path):
        raise ImportError(
            f"{os.path.basename(path)} is not built ({path} missing); run __graft_entry__.build() "
            "first. There is no fallback implementation.")
    lib = ctypes.CDLL(path)
    vp = ctypes.c_void_p
    lib.fa_fwd.restype = ctypes.c_int
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp] + [ctypes.c_int] * 5 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int, vp]
    lib.fa_fwd_ws.restype = ctypes.c_int
    lib.fa_fwd_ws.argtypes = [vp, vp, vp, vp, vp] + [ctypes.c_int] * 5 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_noalloc.restype = ctypes.c_int
    lib.fa_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp] + [ctypes.c_int] * 5 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int, vp]
    lib.fa_fwd_host.restype = ctypes.c_int
    lib.fa_fwd_host.argtypes = [vp, vp, vp, vp, vp] + [ctypes.c_int] * 5 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_host_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_fwd_host_workspace_bytes.argtypes = [ctypes.c_int] * 5
    lib.fa_fwd_dropout.restype = ctypes.c_int
    lib.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp] + [ctypes.c_int] * 5 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_ulonglong,
        ctypes.c_uint, vp]
    lib.fa_fwd_fp8.restype = ctypes.c_int
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp] + [ctypes.c_int] * 5 + [
        ctypes.c_float, ctypes.c_int] + [ctypes.c_float] * 3 + [ctypes.c_int, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_fp8_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_fwd_fp8_workspace_bytes.argtypes = [ctypes.c_int] * 4
    lib.fa_dropout_mask.restype = ctypes.c_int
    lib.fa_dropout_mask.argtypes = [vp] + [ctypes.c_int] * 4 + [
        ctypes.c_float, ctypes.c_ulonglong, ctypes.c_uint, vp]
    lib.fa_bwd.restype = ctypes.c_int
    lib.fa_bwd.argtypes = [vp] * 9 + [ctypes.c_int] * 5 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int, vp, ctypes.c_size_t, vp]
    lib.fa_bwd_dropout.restype = ctypes.c_int
    lib.fa_bwd_dropout.argtypes = [vp] * 9 + [ctypes.c_int] * 5 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_ulonglong,
        ctypes.c_uint, vp, ctypes.c_size_t, vp]
    lib.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_bwd_workspace_bytes.argtypes = [ctypes.c_int] * 5
    lib.fa_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_fwd_workspace_bytes.argtypes = [ctypes.c_int] * 6
    lib.fa_last_status.restype = ctypes.c_int
    lib.fa_last_status.argtypes = []
    lib.fa_stream_status.restype = ctypes.c_int
    lib.fa_stream_status.argtypes = [vp]
    lib.fa_clear_status.restype = ctypes.c_int
    lib.fa_clear_status.argtypes = []
    lib.fa_strerror.restype = ctypes.c_char_p
    lib.fa_strerror.argtypes = [ctypes.c_int]
    lib.fa_selftest_wait_timeout.restype = ctypes.c_int
    lib.fa_selftest_wait_timeout.argtypes = [ctypes.c_int, vp]
    lib.fa_num_kernel_launches.restype = ctypes.c_longlong
    lib.fa_num_kernel_launches.argtypes = []
    lib.fa_set_wait_limit_us.restype = ctypes.c_int
    lib.fa_set_wait_limit_us.argtypes = [ctypes.c_ulonglong]
    lib.fa_get_wait_limit_us.restype = ctypes.c_ulonglong
    lib.fa_get_wait_limit_us.argtypes = []
    heads, kv, rope = ctypes.POINTER(fa_heads), ctypes.POINTER(fa_paged_kv), ctypes.POINTER(fa_rope)
    i, f, n = ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_qk_norm_rope.restype = i
    lib.fa_qk_norm_rope.argtypes = [heads] * 4 + [i, i, i, vp, vp, f, rope, vp, i, vp]
    lib.fa_qk_norm_rope_bwd.restype = i
    lib.fa_qk_norm_rope_bwd.argtypes = [heads] * 6 + [vp, vp, i, i, i, vp, vp, f, rope, vp, i, vp, n, vp]
    lib.fa_qk_norm_rope_bwd_workspace_bytes.restype = n
    lib.fa_qk_norm_rope_bwd_workspace_bytes.argtypes = [i]
    lib.fa_paged_append.restype = i
    lib.fa_paged_append.argtypes = [kv, heads, heads, i, i, vp, vp, vp, i, rope, i, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_fwd_paged.argtypes = [kv, heads, heads, vp, i, i, i, vp, vp, vp, i, f, i, i, vp, n, vp]
    lib.fa_fwd_paged_workspace_bytes.restype = n
    lib.fa_fwd_paged_workspace_bytes.argtypes = [i] * 4
    lib.fa_paged_append_fp8.restype = i
    lib.fa_paged_append_fp8.argtypes = [kv, vp, vp, heads, heads, i, i, vp, vp, vp, i, rope, i, vp]
    lib.fa_fwd_paged_fp8.restype = i
    lib.fa_fwd_paged_fp8.argtypes = [kv, vp, vp, heads, heads, vp, i, i, i, vp, vp, vp, i, f, i, i, vp, n, vp]
    lib.fa_paged_key_weights.restype = i
    lib.fa_paged_key_weights.argtypes = [kv, vp, heads, vp, vp, i, i, i, vp, vp, vp, i, f, i, i, vp]
    lib.fa_paged_evict_workspace_bytes.restype = n
    lib.fa_paged_evict_workspace_bytes.argtypes = [i] * 4
    lib.fa_paged_evict.restype = i
    lib.fa_paged_evict.argtypes = [kv, vp, vp, vp, i, vp, vp, i, i, i, vp, vp, vp, n, vp]
    lib.fa_debug_cap_workspace.restype = ctypes.c_int
    lib.fa_debug_cap_workspace.argtypes = [ctypes.c_longlong]
    return lib


_choice = os.environ.get("FA_LIBRARY", "release")
if _choice not in ("release", "debug"):
    raise ImportError(f"FA_LIBRARY must be 'release' or 'debug', not {_choice!r}")
lib = load_library(DEBUG_LIB_PATH if _choice == "debug" else LIB_PATH)


def strerror(code: int) -> str:
    return lib.fa_strerror(int(code)).decode()


def fa_fwd(Q, K, V, O, L, B, H, Nq, Nk, d, scale, causal, dtype, stream) -> int:
    """Direct C-ABI call with raw integer addresses (device pointers) and sizes."""
    return int(lib.fa_fwd(Q, K, V, O, L, int(B), int(H), int(Nq), int(Nk), int(d),
                          float(scale), int(bool(causal)), int(dtype), stream))


def fa_fwd_ws(Q, K, V, O, L, B, H, Nq, Nk, d, scale, causal, dtype, workspace, workspace_bytes,
              stream) -> int:
    """C-ABI call of the workspace variant (stream-K split of the key range)."""
    return int(lib.fa_fwd_ws(Q, K, V, O, L, int(B), int(H), int(Nq), int(Nk), int(d),
                             float(scale), int(bool(causal)), int(dtype), workspace,
                             int(workspace_bytes), stream))


def fa_fwd_noalloc(Q, K, V, O, L, B, H, Nq, Nk, d, scale, causal, dtype, stream) -> int:
    """C-ABI call of the allocation-free variant (fixed device scratch, see fa_fwd.h)."""
    return int(lib.fa_fwd_noalloc(Q, K, V, O, L, int(B), int(H), int(Nq), int(Nk), int(d),
                                  float(scale), int(bool(causal)), int(dtype), stream))


def fa_fwd_host(Q, K, V, O, L, B, H, Nq, Nk, d, scale, causal, dtype, workspace,
                workspace_bytes, stream) -> int:
    """C-ABI call of the forward pass on HOST buffers (device workspace; see fa_fwd.h)."""
    return int(lib.fa_fwd_host(Q, K, V, O, L, int(B), int(H), int(Nq), int(Nk), int(d),
                               float(scale), int(bool(causal)), int(dtype), workspace,
                               int(workspace_bytes), stream))


def fa_fwd_host_workspace_bytes(B, H, Nq, Nk, d) -> int:
    return int(lib.fa_fwd_host_workspace_bytes(int(B), int(H), int(Nq), int(Nk), int(d)))


def fa_fwd_dropout(Q, K, V, O, L, B, H, Nq, Nk, d, scale, causal, dtype, p_drop, seed, offset,
                   stream) -> int:
    """C-ABI call of the forward pass with dropout (mask of (seed, offset), see fa_fwd.h)."""
    return int(lib.fa_fwd_dropout(Q, K, V, O, L, int(B), int(H), int(Nq), int(Nk), int(d),
                                  float(scale), int(bool(causal)), int(dtype), float(p_drop),
                                  int(seed), int(offset), stream))


def fa_fwd_fp8(Q, K, V, O, L, B, H, Nq, Nk, d, scale, causal, q_descale, k_descale, v_descale,
               out_dtype, workspace, workspace_bytes, stream) -> int:
    """C-ABI call of the E4M3 forward pass (raw device addresses and sizes)."""
    return int(lib.fa_fwd_fp8(Q, K, V, O, L, int(B), int(H), int(Nq), int(Nk), int(d),
                              float(scale), int(bool(causal)), float(q_descale), float(k_descale),
                              float(v_descale), int(out_dtype), workspace, int(workspace_bytes),
                              stream))


def fa_fwd_fp8_workspace_bytes(B, H, Nk, d) -> int:
    return int(lib.fa_fwd_fp8_workspace_bytes(int(B), int(H), int(Nk), int(d)))


def fa_dropout_mask(keep, B, H, Nq, Nk, p_drop, seed, offset, stream) -> int:
    """C-ABI call writing the keep mask [B,H,Nq,Nk] (bytes) of fa_fwd_dropout."""
    return int(lib.fa_dropout_mask(keep, int(B), int(H), int(Nq), int(Nk), float(p_drop),
                                   int(seed), int(offset), stream))


def fa_fwd_workspace_bytes(B, H, Nq, Nk, d, causal) -> int:
    return int(lib.fa_fwd_workspace_bytes(int(B), int(H), int(Nq), int(Nk), int(d),
                                          int(bool(causal))))


def fa_bwd(Q, K, V, O, dO, L, dQ, dK, dV, B, H, Nq, Nk, d, scale, causal, dtype, workspace,
           workspace_bytes, stream) -> int:
    """C-ABI call of the backward pass (raw device addresses and sizes)."""
    return int(lib.fa_bwd(Q, K, V, O, dO, L, dQ, dK, dV, int(B), int(H), int(Nq), int(Nk), int(d),
                          float(scale), int(bool(causal)), int(dtype), workspace,
                          int(workspace_bytes), stream))


def fa_bwd_dropout(Q, K, V, O, dO, L, dQ, dK, dV, B, H, Nq, Nk, d, scale, causal, dtype, p_drop,
                   seed, offset, workspace, workspace_bytes, stream) -> int:
    """C-ABI call of the backward pass of fa_fwd_dropout (same p_drop, seed, offset)."""
    return int(lib.fa_bwd_dropout(Q, K, V, O, dO, L, dQ, dK, dV, int(B), int(H), int(Nq), int(Nk),
                                  int(d), float(scale), int(bool(causal)), int(dtype),
                                  float(p_drop), int(seed), int(offset), workspace,
                                  int(workspace_bytes), stream))


def fa_bwd_workspace_bytes(B, H, Nq, Nk, d) -> int:
    return int(lib.fa_bwd_workspace_bytes(int(B), int(H), int(Nq), int(Nk), int(d)))


def fa_last_status() -> int:
    return int(lib.fa_last_status())


def fa_stream_status(stream=None) -> int:
    """The device-side status once `stream`'s queued work has finished (that stream only)."""
    return int(lib.fa_stream_status(stream))


def fa_clear_status() -> int:
    return int(lib.fa_clear_status())


def fa_selftest_wait_timeout(limit_us: int, stream=None) -> int:
    return int(lib.fa_selftest_wait_timeout(int(limit_us), stream))


def fa_num_kernel_launches() -> int:
    return int(lib.fa_num_kernel_launches())


def fa_set_wait_limit_us(limit_us: int) -> int:
    if not 0 <= int(limit_us) < 1 << 64:
        return FA_ERR_RANGE
    return int(lib.fa_set_wait_limit_us(int(limit_us)))


def fa_get_wait_limit_us() -> int:
    return int(lib.fa_get_wait_limit_us())


def attention(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
              stream=None, workspace=None):
    """O, L = attention(q, k, v) for CUDA tensors q [B,H,Nq,d], k/v [B,H,Nk,d] (fp16/bf16).

    Allocates O (like q) and L ([B,H,Nq] fp32) unless given; launches on `stream`
    (a torch.cuda.Stream, default: the current stream) and returns without synchronising.
    `workspace`: a zero-filled uint8 CUDA tensor of at least fa_fwd_workspace_bytes(...)
    bytes enables the stream-K split for full attention (see include/fa_fwd.h).
    """
    import torch

    # Every check runs before anything touches a device: the kernels write through raw
    # pointers, so a caller-supplied `out`, `lse` or `workspace` of the wrong size, type,
    # layout or device would be written out of bounds.
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("q, k, v must be float16 or bfloat16")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if tuple(k.shape) != (B, H, Nk, d) or tuple(v.shape) != (B, H, Nk, d):
        raise ValueError("k and v must be [B, H, Nk, d] with q's B, H, d")
    if out is not None and (out.dtype != q.dtype or tuple(out.shape) != (B, H, Nq, d)
                            or not out.is_contiguous()):
        raise ValueError("out must be a contiguous [B, H, Nq, d] tensor of q's dtype")
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Nq)
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous [B, H, Nq] float32 tensor")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor")
    tensors = [t for t in (q, k, v, out, lse, workspace) if t is not None]
    if not all(t.is_cuda for t in tensors):
        raise ValueError("q, k, v (and out, lse, workspace when given) must be CUDA tensors")
    if any(t.device != q.device for t in tensors):
        raise ValueError("q, k, v (and out, lse, workspace when given) must be on one device")
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), device=q.device, dtype=torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    dt = FA_BF16 if q.dtype == torch.bfloat16 else FA_F16
    with torch.cuda.device(q.device):
        if workspace is None:
            rc = fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                        B, H, Nq, Nk, d, scale, causal, dt, ctypes.c_void_p(stream.cuda_stream))
        else:
            rc = fa_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           lse.data_ptr(), B, H, Nq, Nk, d, scale, causal, dt,
                           workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                           ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise FAError(rc)
    return out, lse


# ------------------------------------------------------------------ operators of a decoder block
# fa_heads, fa_paged_kv and fa_rope arguments of the C-ABI calls below are the structures above
# (or None for a NULL pointer).
def fa_qk_norm_rope(q, k, q_out, k_out, B, N, d, wq, wk, eps, rope, positions, dtype, stream) -> int:
    """C-ABI call of the per-head norm and position rotation (see fa_decoder.h)."""
    return int(lib.fa_qk_norm_rope(q, k, q_out, k_out, int(B), int(N), int(d), wq, wk, float(eps), rope, positions,
                                   int(dtype), stream))


def fa_qk_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, dwq, dwk, B, N, d, wq, wk, eps, rope, positions, dtype,
                        workspace, workspace_bytes, stream) -> int:
    """C-ABI call of the gradients of fa_qk_norm_rope."""
    return int(lib.fa_qk_norm_rope_bwd(dq_out, dk_out, q, k, dq, dk, dwq, dwk, int(B), int(N), int(d), wq, wk,
                                       float(eps), rope, positions, int(dtype), workspace, int(workspace_bytes),
                                       stream))


def fa_qk_norm_rope_bwd_workspace_bytes(d) -> int:
    return int(lib.fa_qk_norm_rope_bwd_workspace_bytes(int(d)))


def fa_paged_append(kv, k, v, B, T, cu_seqlens, seq_lens, block_table, table_stride, rope, dtype, stream) -> int:
    """C-ABI call writing new keys (rotated) and values into a paged cache."""
    return int(lib.fa_paged_append(kv, k, v, int(B), int(T), cu_seqlens, seq_lens, block_table, int(table_stride),
                                   rope, int(dtype), stream))


def fa_fwd_paged(kv, q, O, L, B, T, max_q, cu_seqlens, seq_lens, block_table, table_stride, scale, causal, dtype,
                 workspace, workspace_bytes, stream) -> int:
    """C-ABI call of attention over a paged cache."""
    return int(lib.fa_fwd_paged(kv, q, O, L, int(B), int(T), int(max_q), cu_seqlens, seq_lens, block_table,
                                int(table_stride), float(scale), int(bool(causal)), int(dtype), workspace,
                                int(workspace_bytes), stream))


def fa_fwd_paged_workspace_bytes(Hq, Hkv, d, max_q) -> int:
    return int(lib.fa_fwd_paged_workspace_bytes(int(Hq), int(Hkv), int(d), int(max_q)))


def fa_paged_append_fp8(kv, k_scale, v_scale, k, v, B, T, cu_seqlens, seq_lens, block_table, table_stride, rope, dtype,
                        stream) -> int:
    """C-ABI call writing new keys (rotated) and values into a paged cache held in 8 bits."""
    return int(lib.fa_paged_append_fp8(kv, k_scale, v_scale, k, v, int(B), int(T), cu_seqlens, seq_lens, block_table,
                                       int(table_stride), rope, int(dtype), stream))


def fa_fwd_paged_fp8(kv, k_scale, v_scale, q, O, L, B, T, max_q, cu_seqlens, seq_lens, block_table, table_stride,
                     scale, causal, dtype, workspace, workspace_bytes, stream) -> int:
    """C-ABI call of attention over a paged cache held in 8 bits."""
    return int(lib.fa_fwd_paged_fp8(kv, k_scale, v_scale, q, O, L, int(B), int(T), int(max_q), cu_seqlens, seq_lens,
                                    block_table, int(table_stride), float(scale), int(bool(causal)), int(dtype),
                                    workspace, int(workspace_bytes), stream))


def fa_paged_key_weights(kv, k_scale, q, L, weights, B, T, max_q, cu_seqlens, seq_lens, block_table, table_stride,
                         scale, causal, dtype, stream) -> int:
    """C-ABI call adding new tokens' attention weights to those of the cached tokens."""
    return int(lib.fa_paged_key_weights(kv, k_scale, q, L, weights, int(B), int(T), int(max_q), cu_seqlens, seq_lens,
                                        block_table, int(table_stride), float(scale), int(bool(causal)), int(dtype),
                                        stream))


def fa_paged_evict(kv, k_scale, v_scale, weights, B, seq_lens, block_table, table_stride, budget, recent, kept,
                   new_lens, workspace, workspace_bytes, stream) -> int:
    """C-ABI call cutting each key head's cached tokens to a budget."""
    return int(lib.fa_paged_evict(kv, k_scale, v_scale, weights, int(B), seq_lens, block_table, int(table_stride),
                                  int(budget), int(recent), kept, new_lens, workspace, int(workspace_bytes), stream))


def fa_paged_evict_workspace_bytes(B, Hkv, budget, held8) -> int:
    return int(lib.fa_paged_evict_workspace_bytes(int(B), int(Hkv), int(budget), int(bool(held8))))


_torch_calls = None


def _calls():
    """The native tensor-level calls (csrc/fa_torch.cpp), bound to the library in use."""
    global _torch_calls
    if _torch_calls is None:
        if not os.path.exists(TORCH_CALLS_PATH):
            raise ImportError(f"{os.path.basename(TORCH_CALLS_PATH)} is not built ({TORCH_CALLS_PATH} missing); run "
                              "__graft_entry__.build() with a CUDA build of torch first. There is no fallback "
                              "implementation.")
        import torch  # noqa: F401  (the module links against libraries that torch loads)

        from . import _fa_torch
        names = ("fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_bytes", "fa_paged_append",
                 "fa_fwd_paged", "fa_fwd_paged_workspace_bytes", "fa_paged_append_fp8", "fa_fwd_paged_fp8",
                 "fa_paged_key_weights", "fa_paged_evict", "fa_paged_evict_workspace_bytes")
        _fa_torch.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names))
        _torch_calls = _fa_torch
    return _torch_calls


def qk_norm_rope(q, k, wq, wk, rope=None, positions=None, eps: float = 1e-6, interleaved: bool = False,
                 q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head and the position rotation, in one pass.

    q [B, N, Hq, d] and k [B, N, Hk, d] (fp16/bf16, d 64 or 128), any strides with adjacent row
    elements, so views of a fused projection serve; wq, wk [d] of the same dtype; rope: fp32
    [length, rot_dim] table (cosines, then sines; see include/fa_decoder.h), None: no rotation;
    positions: int32 [B, N], None: 0 .. N-1 (refused if the table has fewer rows). Returns (q_out, k_out), allocated as contiguous
    [B, N, H, d] unless given (transposed views, and q and k themselves, are allowed).
    Launches on `stream` (a torch.cuda.Stream, default: the current one); what it allocates
    belongs to that stream, and the caller keeps the inputs until that stream is past the call, as
    with torch's own calls on another stream. Not recorded by autograd: in grad mode, inputs that require a gradient
    are refused (qk_norm_rope_backward computes the gradients).
    """
    r = _calls().norm_rope(q, k, wq, wk, rope, positions, eps, interleaved, q_out, k_out, stream)
    if type(r) is int:
        raise FAError(r, "fa_qk_norm_rope")
    return r


def qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, rope=None, positions=None, eps: float = 1e-6,
                          interleaved: bool = False, dq=None, dk=None, stream=None):
    """(dq, dk, dwq, dwk) of qk_norm_rope from its inputs and the gradients of its outputs.

    dq_out [B, N, Hq, d] and dk_out [B, N, Hk, d] with any strides; dq and dk are allocated as
    contiguous [B, N, H, d] unless given; dwq and dwk are fp32 [d].
    """
    r = _calls().norm_rope_backward(dq_out, dk_out, q, k, wq, wk, rope, positions, eps, interleaved, dq, dk, stream)
    if type(r) is int:
        raise FAError(r, "fa_qk_norm_rope_bwd")
    return r


def paged_append(k, v, k_pages, v_pages, block_table, cu_seqlens, seq_lens, rope=None, interleaved: bool = False,
                 stream=None):
    """Writes new keys (rotated by their positions when `rope` is given) and values into a paged cache.

    k, v [T, Hkv, d]; k_pages, v_pages [num_pages, Hkv, page_size, d] with the same strides (a
    transposed view of [num_pages, page_size, Hkv, d] serves); block_table [B, pages], cu_seqlens
    [B + 1] and seq_lens [B] int32: sequence b's new tokens are rows cu_seqlens[b] ..
    cu_seqlens[b+1]-1, the last of its seq_lens[b] positions (see include/fa_decoder.h). In grad
    mode, tensors that require a gradient are refused.
    """
    r = _calls().append(k, v, k_pages, v_pages, block_table, cu_seqlens, seq_lens, rope, interleaved, stream)
    if r != 0:
        raise FAError(r, "fa_paged_append")


def attention_paged(q, k_pages, v_pages, block_table, cu_seqlens, seq_lens, max_q: int, causal: bool = True,
                    scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """O, L of each sequence's new tokens over its paged cache (which holds their keys already).

    q [T, Hq, d], Hq a multiple of the cache's Hkv; the cache and the batch as in paged_append;
    max_q: the most new tokens of a sequence (chooses the kernel). O like q and L [T, Hq] fp32
    are allocated unless given; rows that belong to no sequence are left as they were (in the
    tensors allocated here: uninitialised). `workspace`: a uint8 tensor of at least
    fa_fwd_paged_workspace_bytes(...) bytes, allocated for the call when None. In grad mode, tensors
    that require a gradient are refused.
    """
    r = _calls().attend(q, k_pages, v_pages, block_table, cu_seqlens, seq_lens, max_q, causal, scale, out, lse,
                        workspace, stream)
    if type(r) is int:
        raise FAError(r, "fa_fwd_paged")
    return r


# --------------------------------------------------------------------- a cache held in 8 bits
def paged_append_fp8(k, v, k_pages, v_pages, k_scale, v_scale, block_table, cu_seqlens, seq_lens, rope=None,
                     interleaved: bool = False, stream=None):
    """paged_append for a cache held in 8 bits: k_pages, v_pages float8_e4m3fn [num_pages, Hkv, page_size, d]
    with the same strides (multiples of 16 elements), k_scale, v_scale fp32 [num_pages, Hkv].

    An element is scale * code. A page that gets its first token takes the smallest power of two that
    holds its new tokens; one that has older tokens keeps its scale or, where the new ones need a larger
    one, takes that and its codes are rounded anew (see include/fa_decoder.h).

    `rope` turns a key by its place in the cache. After paged_evict that is not the token's position any more: rotate
    by qk_norm_rope with `positions` and leave `rope` out.
    """
    r = _calls().append_fp8(k, v, k_pages, v_pages, block_table, cu_seqlens, seq_lens, rope, interleaved, stream,
                            k_scale, v_scale)
    if r != 0:
        raise FAError(r, "fa_paged_append_fp8")


def attention_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, cu_seqlens, seq_lens, max_q: int,
                        causal: bool = True, scale: float | None = None, out=None, lse=None, workspace=None,
                        stream=None):
    """attention_paged over a cache held in 8 bits (see paged_append_fp8); q, O (fp16/bf16) and L as there.

    Pages whose v_scale lies far below the largest of their sequence count with fewer bits: with an error of 2^-28 / r of
    their weights at a ratio of r (see include/fa_decoder.h).
    """
    r = _calls().attend_fp8(q, k_pages, v_pages, block_table, cu_seqlens, seq_lens, max_q, causal, scale, out, lse,
                            workspace, stream, k_scale, v_scale)
    if type(r) is int:
        raise FAError(r, "fa_fwd_paged_fp8")
    return r


# ------------------------------------------------------------------------ eviction from a cache
def paged_key_weights(q, lse, k_pages, weights, block_table, cu_seqlens, seq_lens, max_q: int, causal: bool = True,
                      scale: float | None = None, k_scale=None, stream=None):
    """Adds the attention weight that the new tokens give to each cached token to `weights`, in place.

    q [T, Hq, d] and lse [T, Hq] as attention_paged had and returned them; k_pages, the batch, max_q, causal
    and scale as there, k_scale for a cache held in 8 bits; weights: fp32 [num_pages, Hkv, page_size]. A
    new token's own weight starts from 0, whatever stood in its place (see include/fa_decoder.h).
    """
    r = _calls().key_weights(q, lse, k_pages, weights, block_table, cu_seqlens, seq_lens, max_q, causal, scale,
                             k_scale, stream)
    if r != 0:
        raise FAError(r, "fa_paged_key_weights")


def paged_evict(k_pages, v_pages, weights, block_table, seq_lens, budget: int, recent: int, k_scale=None,
                v_scale=None, kept=None, new_lens=None, workspace=None, stream=None):
    """Cuts each key head of every sequence to `budget` cached tokens, in place: the last `recent` and, of
    those before, the ones of the largest weight (see include/fa_decoder.h).

    k_pages, v_pages, weights (and for a cache held in 8 bits k_scale, v_scale) are moved together; seq_lens is
    read. Returns (kept, new_lens): int32 [B, Hkv, budget], the position that each place's token had (-1
    behind the last token of a shorter sequence), and int32 [B], the lengths from now on; allocated unless
    given (new_lens may be seq_lens). `workspace`: a uint8 tensor of at least
    fa_paged_evict_workspace_bytes(...) bytes, allocated for the call when None.

    From then on a cached token's place is not its position: rotate new queries and keys by the tokens' own positions
    (qk_norm_rope with `positions`) and append them without `rope`.
    """
    r = _calls().evict(k_pages, v_pages, weights, block_table, seq_lens, budget, recent, k_scale, v_scale, kept,
                       new_lens, workspace, stream)
    if type(r) is int:
        raise FAError(r, "fa_paged_evict")
    return r
