/* fa_decoder.h -- C ABI of libfa, second part: the operators that stand next to the attention
 * kernels of fa_fwd.h in a decoder block: the norms and the position rotation of the query and
 * key heads (with gradients), a paged cache of keys and values, and attention over that cache.
 *
 * Conventions are those of fa_fwd.h: DEVICE pointers owned by the caller, fp16 or bf16 elements,
 * no allocation, no pointer kept after return, asynchronous on `stream`, host-side argument
 * checks before any CUDA call, FA_ERR_* codes, device-side errors in the status word that
 * fa_last_status() and fa_stream_status() read.
 */
#ifndef FA_DECODER_H
#define FA_DECODER_H

#include "fa_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A set of rows of d elements, one for each (batch, token, head). Element c of the row starts at
 *   ptr + batch*batch_stride + token*token_stride + head*head_stride + c      (in elements):
 * slices of a fused projection, [B, N, H, d] and [B, H, N, d] are all such sets. `ptr` is 16-byte
 * aligned and the strides are multiples of 8 elements; the rows of an output must not overlap. */
typedef struct {
  void* ptr;
  long long batch_stride, token_stride, head_stride;
  int H;
} fa_heads;

/* A paged cache: num_pages pages, each holding page_size tokens of Hkv heads of d elements, for
 * keys and for values (the same strides, in elements, multiples of 8; pointers 16-byte aligned).
 * Row (page, head, slot) starts at page*page_stride + head*head_stride + slot*token_stride, so
 * [pages, Hkv, page_size, d] and [pages, page_size, Hkv, d] are both such caches.
 * page_size is 8, 16, 32, 64 or a multiple of 128.
 *
 * A batch of B sequences (at most 2^30) over such a cache is given by int32 device arrays:
 *   cu_seqlens  [B + 1]  new tokens cu_seqlens[b] .. cu_seqlens[b+1]-1 of the T packed token rows
 *                        belong to sequence b (a sequence may have none); rows before the first
 *                        and behind the last sequence are neither read nor written
 *   seq_lens    [B]      tokens of sequence b in the cache, the new ones counted
 *   block_table [B, table_stride]  entry i of row b: the page of tokens i*page_size ...; at least
 *                        ceil(seq_lens[b] / page_size) valid entries, others are not used.
 * New token i of the n of sequence b stands at position seq_lens[b] - n + i. */
typedef struct {
  void *k, *v;
  long long page_stride, head_stride, token_stride;
  int num_pages, page_size, Hkv, d;
} fa_paged_kv;

/* A rotation table: fp32 [length, rot_dim], 16-byte aligned; row p holds the cosines of position
 * p's rot_dim/2 angles, then their sines. The rotation turns the first rot_dim elements of a row
 * (a multiple of 16, at most d; the others pass through), pair i by angle i: elements
 * (i, i + rot_dim/2), or (2i, 2i+1) if `interleaved`:
 *   (a, b) -> (a cos - b sin, b cos + a sin).
 * A NULL table (or a NULL fa_rope) means no rotation. */
typedef struct {
  const float* table;
  int length, rot_dim, interleaved;
} fa_rope;

/* fa_qk_norm_rope -- RMS norm of every query and key head, then the rotation, in one pass:
 *     y = R(position) (x * r * w),   r = (mean_c x_c^2 + eps)^(-1/2)
 * for the rows x of q (weights wq) and of k (weights wk).
 *   q, k          inputs [B, N, H] of d elements; H may be 0 for one of them (it is then skipped
 *                 and its pointers are not looked at)
 *   q_out, k_out  outputs; may be the same memory as the inputs with the same strides (in place)
 *   wq, wk        [d] weights, `dtype`, 16-byte aligned
 *   positions     int32 [B, N] rows of the table, or NULL for position n of row n (the table then
 *                 has at least N rows, or the call is refused with FA_ERR_RANGE)
 *   d 64 or 128; eps >= 0 and finite
 * Sums and products are fp32, rounded once (so a row whose mean square passes the range of fp32 comes
 * out as zeros, and with eps = 0 a row of zeros as NaN). A position outside the table records FA_ERR_RANGE in
 * the status word; that token's outputs are left as they were. One kernel. B, N == 0: no-op.
 *
 * fa_qk_norm_rope_bwd -- its gradients, from the same inputs and the gradients dq_out, dk_out of
 * the outputs: with g = R^T dy, u = g * w,
 *     dx = r (u - x r mean_c(u x r)),   dw = sum over all rows of g * x * r
 *   dq, dk        outputs (dq may be dq_out's own memory with the same strides)
 *   dwq, dwk      [d] fp32 outputs; a set with H == 0 leaves its own unwritten. A token whose
 *                 position is out of range adds nothing to them.
 *   workspace     fa_qk_norm_rope_bwd_workspace_bytes(d) bytes, 16-byte aligned, no initialisation
 * Two kernels; no atomics on results, so they do not change from run to run. */
int fa_qk_norm_rope(const fa_heads* q, const fa_heads* k, const fa_heads* q_out, const fa_heads* k_out,
                    int B, int N, int d, const void* wq, const void* wk, float eps,
                    const fa_rope* rope, const int* positions, fa_dtype dtype, void* stream);
size_t fa_qk_norm_rope_bwd_workspace_bytes(int d);
int fa_qk_norm_rope_bwd(const fa_heads* dq_out, const fa_heads* dk_out, const fa_heads* q,
                        const fa_heads* k, const fa_heads* dq, const fa_heads* dk, float* dwq,
                        float* dwk, int B, int N, int d, const void* wq, const void* wk, float eps,
                        const fa_rope* rope, const int* positions, fa_dtype dtype, void* workspace,
                        size_t workspace_bytes, void* stream);

/* fa_paged_append -- write the new tokens' keys and values into the cache, the keys rotated by
 * their positions (no rotation without a table: a plain copy).
 *   kv      the cache; kv->d 64 or 128
 *   k, v    [T, Hkv] rows of d elements (batch_stride unused), dtype as the cache
 *   B, T    sequences, and token rows behind k and v
 * Two new tokens never share a slot as long as no page stands twice in the tables of sequences
 * that are being written. A token whose position is negative, past the table's width or the
 * rotation table, or whose page is not in [0, num_pages) is skipped and FA_ERR_RANGE recorded in
 * the status word. So is a sequence whose rows do not lie in [0, T]; where cu_seqlens decreases, other
 * sequences' tokens may be skipped with it, and nothing is written but a sequence's own tokens in
 * their own places. One kernel. B or T == 0: no-op. */
int fa_paged_append(const fa_paged_kv* kv, const fa_heads* k, const fa_heads* v, int B, int T,
                    const int* cu_seqlens, const int* seq_lens, const int* block_table,
                    int table_stride, const fa_rope* rope, fa_dtype dtype, void* stream);

/* A table of at most this many keys per sequence (table_stride * page_size) needs no workspace. */
#define FA_PAGED_WHOLE_KEYS 512

/* fa_fwd_paged -- attention of each sequence's new tokens over its cache (which already holds
 * their own keys and values). Query head h reads key head h / (Hq / Hkv); Hq is a multiple of
 * Hkv, at most 128 * Hkv.
 *     s_j = scale <q, k_j>,  j in [0, seq_lens[b]), and with `causal` j <= the token's position
 *     O = sum_j softmax_j(s) v_j,   L = ln sum_j exp(s_j)
 * A row that sees no key (an empty sequence, or a negative position) gets O = 0 and L = -inf,
 * whatever its query holds. A row that sees keys and whose scores hold a NaN, or pass the range of
 * fp32, gets NaN in O, and in L the NaN (or -inf where every score lies below that range).
 *   q, O      [T, Hq] rows of d elements (batch_stride unused); kv->d 64 or 128. O may be q's own
 *             memory with the same strides
 *   L         fp32 [T, Hq], or NULL
 *   max_q     the most new tokens that a sequence of this batch has: it chooses the kernel and
 *             sizes the workspace; a larger batch still gets right results, more slowly. >= 1
 *   workspace fa_fwd_paged_workspace_bytes() bytes on the current device, 256-byte aligned, no
 *             initialisation; calls that share one must not overlap on the GPU. Not used, and may
 *             be NULL, when table_stride * page_size <= FA_PAGED_WHOLE_KEYS
 * The key ranges of all sequences are cut into equal shares for the SMs on the device, from the
 * arrays at the time the kernels run, so a captured call may be replayed with other lengths (up
 * to max_q, B, T and the table's width). Results do not change from run to run.
 * Whatever cached rows hold that no query of the batch sees (the rest of a sequence's last page,
 * pages it does not use) does not matter, NaN included; the keys and values of every position
 * below seq_lens must be finite.
 * A length past the table's width is cut to it, a page outside [0, num_pages) reads as zeros;
 * either records FA_ERR_RANGE in the status word. Two kernels (one without a workspace).
 * A sequence whose rows do not lie in [0, T] is passed over and FA_ERR_RANGE recorded; a negative
 * length counts as zero.
 * Errors as fa_fwd: FA_ERR_NULL, FA_ERR_HEAD_DIM, FA_ERR_SHAPE, FA_ERR_SCALE, FA_ERR_ALIGN,
 * FA_ERR_DTYPE, FA_ERR_WORKSPACE, FA_ERR_TENSOR_MAP for strides that TMA cannot walk (zero or
 * negative along an axis of more than one element, 2^40 bytes and more), and FA_ERR_RANGE for a
 * page size that is not allowed. */
size_t fa_fwd_paged_workspace_bytes(int Hq, int Hkv, int d, int max_q);
int fa_fwd_paged(const fa_paged_kv* kv, const fa_heads* q, const fa_heads* O, float* L, int B, int T,
                 int max_q, const int* cu_seqlens, const int* seq_lens, const int* block_table,
                 int table_stride, float scale, int causal, fa_dtype dtype, void* workspace,
                 size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_DECODER_H */
