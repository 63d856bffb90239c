// fa_decoder.cu -- the C ABI of include/fa_decoder.h: argument checks and launches. The kernels
// live in fa_rope.cuh (norm, rotation, append) and fa_paged.cuh (attention over a paged cache).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "fa_decoder_host.h"

namespace {

using namespace fa;
using namespace fa_decoder;

// How the (token, head) rows are shared out: a group of d/8 lanes walks `chunk` heads of a token,
// all of them (the token's angles and addresses are then worked out once), or fewer while the
// tokens alone do not give the SMs enough warps to cover the memory latency: ROW_MIN_WARPS = 16 per
// SM (1000 tokens of 32 + 8 heads, d 128, forward: 5.2 us, with 8 warps 6.5, with 32 6.1; 4000 tokens
// 14.2, 21.9, 16.5; their gradients: 1000 tokens 12.5, 9.8, 12.2, 4000 tokens 32.3 with any of them).
struct RowShare {
  int chunk, n_chunks;
  uint32_t units;  // warps
};
// `walked`: a fixed number of blocks walks the units (the backward pass). Its last round is then a
// smaller part of the whole with more units: 94 -> 88 us for 16384 tokens of 32 + 8 heads, d = 128 (3
// and 12 times ROW_MIN_WARPS instead of 6: 94 and 101), 60.4 -> 57.4 of 12 + 12; but 28.3 -> 32.3 us for
// 4000 tokens of 32 + 8. With fewer than 8 heads to a unit it costs more than it gives.
RowShare share_rows(long long tokens, int heads, int d, int sms, bool walked) {
  const int groups = 256 / d;  // of lanes in a warp
  const long long warps = (tokens + groups - 1) / groups;
  RowShare r;
  r.chunk = heads;
  auto fewer_than = [&](int per_sm) { return warps * ((heads + r.chunk - 1) / r.chunk) < (long long)sms * per_sm; };
  while (r.chunk > 1 && fewer_than(ROW_MIN_WARPS)) r.chunk = (r.chunk + 1) / 2;
  while (walked && r.chunk >= 16 && fewer_than(6 * ROW_MIN_WARPS)) r.chunk = (r.chunk + 1) / 2;
  r.n_chunks = (heads + r.chunk - 1) / r.chunk;
  r.units = (uint32_t)(warps * r.n_chunks);
  return r;
}

int norm_rope_args(const fa_heads* const* sets, int n, int B, int N, int d, const void* wq, const void* wk,
                   float eps, const fa_rope* rope, const int* positions, fa_dtype dtype, bool* noop) {
  *noop = false;
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (d != 64 && d != 128) return FA_ERR_HEAD_DIM;
  if (B < 0 || N < 0) return FA_ERR_SHAPE;
  if (!(eps >= 0.f) || !isfinite(eps)) return FA_ERR_RANGE;
  int rc = check_rope(rope, d);
  if (rc != FA_OK) return rc;
  for (int i = 0; i < n; ++i)
    if (!sets[i]) return FA_ERR_NULL;
  const int Hq = sets[0]->H, Hk = sets[1]->H;
  for (int i = 0; i < n; ++i)  // q, k, q, k, ...
    if (sets[i]->H != (i & 1 ? Hk : Hq)) return FA_ERR_SHAPE;
  if (Hq < 0 || Hk < 0 || (long long)Hq + Hk > 0x7fffffffLL) return FA_ERR_SHAPE;
  if (B == 0 || N == 0 || Hq + Hk == 0) { *noop = true; return FA_OK; }
  // token n without a position of its own takes row n of the table
  if (rope && rope->table && rope->rot_dim && !positions && N > rope->length) return FA_ERR_RANGE;
  const long long tokens = (long long)B * N;
  if (tokens > 0x7fffffffLL || tokens * ((long long)Hq + Hk) > 0x7fffffffLL) return FA_ERR_SHAPE;
  for (int i = 0; i < n; ++i)
    if ((rc = check_heads(sets[i])) != FA_OK) return rc;
  if ((Hq && !wq) || (Hk && !wk)) return FA_ERR_NULL;
  if ((Hq && !aligned16(wq)) || (Hk && !aligned16(wk)) || !aligned4(positions)) return FA_ERR_ALIGN;
  return FA_OK;
}

NormRopeParams norm_rope_params(const fa_heads* q, const fa_heads* k, const fa_heads* qo, const fa_heads* ko, int B,
                                int N, const void* wq, const void* wk, float eps, const fa_rope* rope,
                                const int* positions) {
  NormRopeParams p = {};
  p.x[0] = dev(q);
  p.x[1] = dev(k);
  p.y[0] = dev(qo);
  p.y[1] = dev(ko);
  p.w[0] = static_cast<const uint16_t*>(wq);
  p.w[1] = static_cast<const uint16_t*>(wk);
  p.eps = eps;
  p.rope = dev(rope);
  p.positions = positions;
  p.N = N;
  return p;
}

void row_units(NormRopeParams* p, long long tokens, int heads, int d, int sms, bool walked) {
  const RowShare r = share_rows(tokens, heads, d, sms, walked);
  p->tokens = (int)tokens;
  p->chunk = r.chunk;
  p->n_chunks = r.n_chunks;
  p->units = r.units;
}

}  // namespace

extern "C" {

int fa_qk_norm_rope(const fa_heads* q, const fa_heads* k, const fa_heads* q_out, const fa_heads* k_out, int B,
                    int N, int d, const void* wq, const void* wk, float eps, const fa_rope* rope,
                    const int* positions, fa_dtype dtype, void* stream) {
  const fa_heads* sets[4] = {q, k, q_out, k_out};
  bool noop = false;
  int rc = norm_rope_args(sets, 4, B, N, d, wq, wk, eps, rope, positions, dtype, &noop);
  if (rc != FA_OK || noop) return rc;
  int index = 0, sms = 0;
  if ((rc = fa_host::current_device(&index, &sms)) != FA_OK) return rc;
  NormRopeParams p = norm_rope_params(q, k, q_out, k_out, B, N, wq, wk, eps, rope, positions);
  if ((rc = fa_host::status_word(&p.status)) != FA_OK) return rc;
  const int H = q->H + k->H;
  row_units(&p, (long long)B * N, H, d, sms, false);
  const unsigned grid = (p.units - 1) / ROW_WARPS + 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return by_type(dtype, rope, d, [&](auto bf, auto inter, auto full) {
    return launch_dependent(d == 64 ? fa_norm_rope_kernel<64, bf, inter, full> : fa_norm_rope_kernel<128, bf, inter, full>,
                            dim3(grid), dim3(ROW_THREADS), 0, st, p);
  });
}

size_t fa_qk_norm_rope_bwd_workspace_bytes(int d) {
  return d == 64 || d == 128 ? (size_t)ROW_BWD_MAX_BLOCKS * 2 * d * sizeof(float) : 0;
}

int fa_qk_norm_rope_bwd(const fa_heads* dq_out, const fa_heads* dk_out, const fa_heads* q, const fa_heads* k,
                        const fa_heads* dq, const fa_heads* dk, float* dwq, float* dwk, int B, int N, int d,
                        const void* wq, const void* wk, float eps, const fa_rope* rope, const int* positions,
                        fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const fa_heads* sets[6] = {dq_out, dk_out, q, k, dq, dk};
  bool noop = false;
  int rc = norm_rope_args(sets, 6, B, N, d, wq, wk, eps, rope, positions, dtype, &noop);
  if (rc != FA_OK) return rc;
  if ((q->H && !dwq) || (k->H && !dwk)) return FA_ERR_NULL;
  if (!aligned4(dwq) || !aligned4(dwk)) return FA_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (noop) {  // no rows: the weights' gradients are sums over nothing
    if (q->H && cudaMemsetAsync(dwq, 0, d * sizeof(float), st) != cudaSuccess) return FA_ERR_CUDA;
    if (k->H && cudaMemsetAsync(dwk, 0, d * sizeof(float), st) != cudaSuccess) return FA_ERR_CUDA;
    return FA_OK;
  }
  if (!workspace || workspace_bytes < fa_qk_norm_rope_bwd_workspace_bytes(d)) return FA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FA_ERR_ALIGN;
  int index = 0, sms = 0;
  if ((rc = fa_host::current_device(&index, &sms)) != FA_OK) return rc;
  NormRopeParams p = norm_rope_params(q, k, dq, dk, B, N, wq, wk, eps, rope, positions);
  if ((rc = fa_host::status_word(&p.status)) != FA_OK) return rc;
  p.g[0] = dev(dq_out);
  p.g[1] = dev(dk_out);
  p.part = static_cast<float*>(workspace);
  const int H = q->H + k->H;
  row_units(&p, (long long)B * N, H, d, sms, true);
  const int most = 2 * sms < ROW_BWD_MAX_BLOCKS ? 2 * sms : ROW_BWD_MAX_BLOCKS;
  const unsigned blocks = (p.units - 1) / ROW_WARPS + 1;
  const int grid = blocks < (unsigned)most ? (int)blocks : most;
  float* oq = q->H ? dwq : nullptr;
  float* ok = k->H ? dwk : nullptr;
  return by_type(dtype, rope, d, [&](auto bf, auto inter, auto full) {
    const int rc1 = launch_dependent(
        d == 64 ? fa_norm_rope_bwd_kernel<64, bf, inter, full> : fa_norm_rope_bwd_kernel<128, bf, inter, full>,
        dim3(grid), dim3(ROW_THREADS), 0, st, p);
    if (rc1 != FA_OK) return rc1;
    return launch_dependent(d == 64 ? fa_norm_rope_dw_kernel<64> : fa_norm_rope_dw_kernel<128>, dim3(2 * d / 32),
                            dim3(32, 32), 0, st, (const float*)p.part, grid, oq, ok);
  });
}

int fa_paged_append(const fa_paged_kv* kv, const fa_heads* k, const fa_heads* v, int B, int T, const int* cu_seqlens,
                    const int* seq_lens, const int* block_table, int table_stride, const fa_rope* rope,
                    fa_dtype dtype, void* stream) {
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (!kv || !k || !v) return FA_ERR_NULL;
  int rc = check_kv(kv);
  if (rc != FA_OK) return rc;
  if (B < 0 || T < 0 || table_stride < 0 || k->H != kv->Hkv || v->H != kv->Hkv) return FA_ERR_SHAPE;
  if ((rc = check_rope(rope, kv->d)) != FA_OK) return rc;
  if (B == 0 || T == 0 || kv->Hkv == 0) return FA_OK;
  if ((long long)T * 2 * kv->Hkv > 0x7fffffffLL || B > MAX_SEQUENCES) return FA_ERR_SHAPE;
  if ((rc = check_heads(k)) != FA_OK || (rc = check_heads(v)) != FA_OK) return rc;
  if (!cu_seqlens || !seq_lens || (!block_table && table_stride)) return FA_ERR_NULL;
  if (!aligned4(cu_seqlens) || !aligned4(seq_lens) || !aligned4(block_table)) return FA_ERR_ALIGN;
  int index = 0, sms = 0;
  if ((rc = fa_host::current_device(&index, &sms)) != FA_OK) return rc;
  AppendParams p = {};
  if ((rc = fa_host::status_word(&p.status)) != FA_OK) return rc;
  p.k = dev(k);
  p.v = dev(v);
  p.kp = static_cast<uint16_t*>(kv->k);
  p.vp = static_cast<uint16_t*>(kv->v);
  p.page_stride = kv->page_stride;
  p.head_stride = kv->head_stride;
  p.token_stride = kv->token_stride;
  p.num_pages = kv->num_pages;
  p.page_size = kv->page_size;
  p.cu = cu_seqlens;
  p.lens = seq_lens;
  p.table = block_table;
  p.table_stride = table_stride;
  p.B = B;
  p.T = T;
  p.rope = dev(rope);
  const RowShare r = share_rows(T, 2 * kv->Hkv, kv->d, sms, false);
  p.chunk = r.chunk;
  p.n_chunks = r.n_chunks;
  p.units = r.units;
  const unsigned grid = (p.units - 1) / ROW_WARPS + 2;  // the last block looks over cu_seqlens
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return by_type(dtype, rope, kv->d, [&](auto bf, auto inter, auto full) {
    return launch_dependent(
        kv->d == 64 ? fa_paged_append_kernel<64, bf, inter, full> : fa_paged_append_kernel<128, bf, inter, full>,
        dim3(grid), dim3(ROW_THREADS), 0, st, p);
  });
}

size_t fa_fwd_paged_workspace_bytes(int Hq, int Hkv, int d, int max_q) {
  int index = 0, sms = 0;
  if ((d != 64 && d != 128) || Hkv <= 0 || Hq <= 0 || Hq % Hkv || Hq / Hkv > 128 || max_q < 1) return 0;
  if (fa_host::current_device(&index, &sms) != FA_OK) return 0;
  return paged_records_bytes(sms) + paged_parts_bytes(sms, d, paged_form(Hq / Hkv, max_q));
}

int fa_fwd_paged(const fa_paged_kv* kv, const fa_heads* q, const fa_heads* O, float* L, int B, int T, int max_q,
                 const int* cu_seqlens, const int* seq_lens, const int* block_table, int table_stride, float scale,
                 int causal, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return attend_paged<false>(kv, nullptr, nullptr, q, O, L, B, T, max_q, cu_seqlens, seq_lens, block_table,
                             table_stride, scale, causal, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
