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
``paged_append`` and ``attention_paged``.
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


def _type_code(t, what):
    import torch

    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_F16
    raise TypeError(f"{what} must be float16 or bfloat16")


def _heads(t, what, dtype, shape=None, written=False):
    """fa_heads of a [..., tokens, heads, d] tensor (3 or 4 dimensions)."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must have the other tensors' dtype")
    size, stride = t.shape, t.stride()
    if shape is not None and tuple(size) != tuple(shape):
        raise ValueError(f"{what} must be {list(shape)}, not {list(size)}")
    if stride[-1] != 1 and size[-1] > 1:
        raise ValueError(f"the elements of a row of {what} must be adjacent (stride 1)")
    # the stride of an axis of one element is never used, and torch may report any
    s = [0 if n <= 1 else st for n, st in zip(size[:-1], stride)]
    if written and any(n > 1 and st == 0 for n, st in zip(size[:-1], s)):
        raise ValueError(f"the rows of {what} must not overlap")
    if len(s) == 2:
        s.insert(0, 0)
    return fa_heads(t.data_ptr(), s[0], s[1], s[2], size[-2])


def _on_device(tensors):
    """Every tensor (None: not given) is a CUDA tensor on the first one's device."""
    dev = tensors[0].device
    for t in tensors:
        if t is not None and (t.device != dev or not t.is_cuda):
            raise ValueError("the tensors must be CUDA tensors on one device")
    return dev


def _index(t, what, shape):
    import torch

    if t.dtype != torch.int32:
        raise TypeError(f"{what} must be int32")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {list(shape)}, not {list(t.shape)}")
    return t.data_ptr()


def _rope(rope, interleaved, d):
    """fa_rope of a [length, rot_dim] fp32 table; None for none."""
    import torch

    if rope is None:
        return None
    if rope.dtype != torch.float32:
        raise TypeError("rope must be float32")
    if rope.dim() != 2 or not rope.is_contiguous() or rope.shape[1] % 16 or rope.shape[1] > d:
        raise ValueError("rope must be a contiguous [length, rot_dim] table, rot_dim a multiple of 16 up to d")
    return fa_rope(rope.data_ptr(), rope.shape[0], rope.shape[1], int(bool(interleaved)))


def _cache(k_pages, v_pages, dtype):
    """fa_paged_kv of [num_pages, Hkv, page_size, d] tensors with the same strides."""
    if k_pages.dtype != dtype or v_pages.dtype != dtype:
        raise TypeError("the cache must have the other tensors' dtype")
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must both be [num_pages, Hkv, page_size, d]")
    size, ks, vs = k_pages.shape, k_pages.stride(), v_pages.stride()
    if any(n > 1 and a != b for n, a, b in zip(size, ks, vs)):
        raise ValueError("k_pages and v_pages must have the same strides")
    if ks[3] != 1 and size[3] > 1:
        raise ValueError("the elements of a cached row must be adjacent (stride 1)")
    s = [0 if n <= 1 else a for n, a in zip(size, ks)]
    return fa_paged_kv(k_pages.data_ptr(), v_pages.data_ptr(), s[0], s[1], s[2], size[0], size[2], size[1], size[3])


def _table(block_table, B):
    """(pointer, width) of a [B, width] int32 table."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, pages per sequence]")
    return _index(block_table, "block_table", (B, block_table.shape[1])), block_table.shape[1]


class _Launch:
    """The device and stream of a call: what is allocated inside belongs to that stream."""

    def __init__(self, device, stream):
        import torch

        self.device = torch.cuda.device(device)
        self.inner = None if stream is None else torch.cuda.stream(stream)
        self.stream = stream or torch.cuda.current_stream(device)

    def __enter__(self):
        self.device.__enter__()
        if self.inner is not None:
            self.inner.__enter__()
        return ctypes.c_void_p(self.stream.cuda_stream)

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)
        self.device.__exit__(*exc)


def qk_norm_rope(q, k, wq, wk, rope=None, positions=None, eps: float = 1e-6, interleaved: bool = False,
                 q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head and the position rotation, in one pass.

    q [B, N, Hq, d] and k [B, N, Hk, d] (fp16/bf16, d 64 or 128), any strides with adjacent row
    elements, so views of a fused projection serve; wq, wk [d] of the same dtype; rope: fp32
    [length, rot_dim] table (cosines, then sines; see include/fa_decoder.h), None: no rotation;
    positions: int32 [B, N], None: 0 .. N-1. Returns (q_out, k_out), allocated as contiguous
    [B, N, H, d] unless given (transposed views, and q and k themselves, are allowed).
    """
    import torch

    dt = _type_code(q, "q and k")
    if q.dim() != 4 or k.dim() != 4 or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError("q and k must be [B, N, H, d] with the same B, N and d")
    B, N, _, d = q.shape
    hq, hk = _heads(q, "q", q.dtype), _heads(k, "k", q.dtype)
    if wq.dtype != q.dtype or wk.dtype != q.dtype:
        raise TypeError("wq and wk must have q's dtype")
    if tuple(wq.shape) != (d,) or tuple(wk.shape) != (d,) or not wq.is_contiguous() or not wk.is_contiguous():
        raise ValueError("wq and wk must be contiguous [d]")
    rp = _rope(rope, interleaved, d)
    pos = None if positions is None else _index(positions, "positions", (B, N))
    oq = None if q_out is None else _heads(q_out, "q_out", q.dtype, q.shape, written=True)
    ok = None if k_out is None else _heads(k_out, "k_out", q.dtype, k.shape, written=True)
    dev = _on_device((q, k, wq, wk, rope, positions, q_out, k_out))
    with _Launch(dev, stream) as st:
        if oq is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            oq = _heads(q_out, "q_out", q.dtype)
        if ok is None:
            k_out = torch.empty(k.shape, dtype=q.dtype, device=dev)
            ok = _heads(k_out, "k_out", q.dtype)
        rc = fa_qk_norm_rope(hq, hk, oq, ok, B, N, d, wq.data_ptr(), wk.data_ptr(), eps, rp, pos, dt, st)
    if rc != 0:
        raise FAError(rc, "fa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, wq, wk, rope=None, positions=None, eps: float = 1e-6,
                          interleaved: bool = False, dq=None, dk=None, stream=None):
    """(dq, dk, dwq, dwk) of qk_norm_rope from its inputs and the gradients of its outputs.

    dq_out [B, N, Hq, d] and dk_out [B, N, Hk, d] with any strides; dq and dk are allocated as
    contiguous [B, N, H, d] unless given; dwq and dwk are fp32 [d].
    """
    import torch

    dt = _type_code(q, "q and k")
    if q.dim() != 4 or k.dim() != 4 or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError("q and k must be [B, N, H, d] with the same B, N and d")
    B, N, _, d = q.shape
    hq, hk = _heads(q, "q", q.dtype), _heads(k, "k", q.dtype)
    gq, gk = _heads(dq_out, "dq_out", q.dtype, q.shape), _heads(dk_out, "dk_out", q.dtype, k.shape)
    if wq.dtype != q.dtype or wk.dtype != q.dtype:
        raise TypeError("wq and wk must have q's dtype")
    if tuple(wq.shape) != (d,) or tuple(wk.shape) != (d,) or not wq.is_contiguous() or not wk.is_contiguous():
        raise ValueError("wq and wk must be contiguous [d]")
    rp = _rope(rope, interleaved, d)
    pos = None if positions is None else _index(positions, "positions", (B, N))
    oq = None if dq is None else _heads(dq, "dq", q.dtype, q.shape, written=True)
    ok = None if dk is None else _heads(dk, "dk", q.dtype, k.shape, written=True)
    dev = _on_device((q, k, wq, wk, rope, positions, dq_out, dk_out, dq, dk))
    with _Launch(dev, stream) as st:
        if oq is None:
            dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
            oq = _heads(dq, "dq", q.dtype)
        if ok is None:
            dk = torch.empty(k.shape, dtype=q.dtype, device=dev)
            ok = _heads(dk, "dk", q.dtype)
        dw = torch.zeros(2, d, dtype=torch.float32, device=dev) if 0 in (hq.H, hk.H) else torch.empty(
            2, d, dtype=torch.float32, device=dev)
        nws = fa_qk_norm_rope_bwd_workspace_bytes(d)
        ws = torch.empty(nws, dtype=torch.uint8, device=dev)
        rc = fa_qk_norm_rope_bwd(gq, gk, hq, hk, oq, ok, dw.data_ptr(), dw.data_ptr() + 4 * d, B, N, d,
                                 wq.data_ptr(), wk.data_ptr(), eps, rp, pos, dt, ws.data_ptr(), nws, st)
    if rc != 0:
        raise FAError(rc, "fa_qk_norm_rope_bwd")
    return dq, dk, dw[0], dw[1]


def paged_append(k, v, k_pages, v_pages, block_table, cu_seqlens, seq_lens, rope=None, interleaved: bool = False,
                 stream=None):
    """Writes new keys (rotated by their positions when `rope` is given) and values into a paged cache.

    k, v [T, Hkv, d]; k_pages, v_pages [num_pages, Hkv, page_size, d] with the same strides (a
    transposed view of [num_pages, page_size, Hkv, d] serves); block_table [B, pages], cu_seqlens
    [B + 1] and seq_lens [B] int32: sequence b's new tokens are rows cu_seqlens[b] ..
    cu_seqlens[b+1]-1, the last of its seq_lens[b] positions (see include/fa_decoder.h).
    """
    dt = _type_code(k, "k and v")
    if k.dim() != 3:
        raise ValueError("k and v must be [T, Hkv, d]")
    hk, hv = _heads(k, "k", k.dtype), _heads(v, "v", k.dtype, k.shape)
    kv = _cache(k_pages, v_pages, k.dtype)
    T, Hkv, d = k.shape
    if (kv.Hkv, kv.d) != (Hkv, d):
        raise ValueError("the cache must have k's heads and head dimension")
    B = seq_lens.shape[0]
    lens, cu = _index(seq_lens, "seq_lens", (B,)), _index(cu_seqlens, "cu_seqlens", (B + 1,))
    table, width = _table(block_table, B)
    rp = _rope(rope, interleaved, d)
    dev = _on_device((k, v, k_pages, v_pages, block_table, cu_seqlens, seq_lens, rope))
    with _Launch(dev, stream) as st:
        rc = fa_paged_append(kv, hk, hv, B, T, cu, lens, table, width, rp, dt, st)
    if rc != 0:
        raise FAError(rc, "fa_paged_append")


def attention_paged(q, k_pages, v_pages, block_table, cu_seqlens, seq_lens, max_q: int, causal: bool = True,
                    scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """O, L of each sequence's new tokens over its paged cache (which holds their keys already).

    q [T, Hq, d], Hq a multiple of the cache's Hkv; the cache and the batch as in paged_append;
    max_q: the most new tokens of a sequence (chooses the kernel). O like q and L [T, Hq] fp32
    are allocated unless given; rows that belong to no sequence are left as they were (in the
    tensors allocated here: uninitialised). `workspace`: a uint8 tensor of at least
    fa_fwd_paged_workspace_bytes(...) bytes, allocated for the call when None.
    """
    import torch

    dt = _type_code(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, d]")
    T, Hq, d = q.shape
    hq = _heads(q, "q", q.dtype)
    kv = _cache(k_pages, v_pages, q.dtype)
    if kv.d != d:
        raise ValueError("the cache must have q's head dimension")
    B = seq_lens.shape[0]
    lens, cu = _index(seq_lens, "seq_lens", (B,)), _index(cu_seqlens, "cu_seqlens", (B + 1,))
    table, width = _table(block_table, B)
    ho = None if out is None else _heads(out, "out", q.dtype, q.shape, written=True)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (T, Hq) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous [T, Hq] float32 tensor")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor")
    dev = _on_device((q, k_pages, v_pages, block_table, cu_seqlens, seq_lens, out, lse, workspace))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _Launch(dev, stream) as st:
        if ho is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            ho = _heads(out, "out", q.dtype)
        if lse is None:
            lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(max(1, fa_fwd_paged_workspace_bytes(Hq, kv.Hkv, d, max_q)), dtype=torch.uint8,
                                    device=dev)
        rc = fa_fwd_paged(kv, hq, ho, lse.data_ptr(), B, T, max_q, cu, lens, table, width, scale, causal, dt,
                          workspace.data_ptr(), workspace.numel(), st)
    if rc != 0:
        raise FAError(rc, "fa_fwd_paged")
    return out, lse
