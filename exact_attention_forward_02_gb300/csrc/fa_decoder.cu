// fa_decoder.cu -- the C ABI of include/fa_decoder.h: argument checks and launches. The kernels
// live in fa_rope.cuh (norm, rotation, append) and fa_paged.cuh (attention over a paged cache).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "fa_decoder.h"
#include "fa_host.h"
#include "fa_paged.cuh"
#include "fa_rope.cuh"

namespace {

using namespace fa;

bool aligned16(const void* ptr) { return ((uintptr_t)ptr & 15) == 0; }
bool aligned4(const void* ptr) { return ((uintptr_t)ptr & 3) == 0; }

// Checks of one set of rows; a set with H == 0 passes.
int check_heads(const fa_heads* h) {
  if (h->H < 0) return FA_ERR_SHAPE;
  if (h->H == 0) return FA_OK;
  if (!h->ptr) return FA_ERR_NULL;
  if (!aligned16(h->ptr) || ((h->batch_stride | h->token_stride | h->head_stride) & 7)) return FA_ERR_ALIGN;
  return FA_OK;
}

int check_rope(const fa_rope* r, int d) {
  if (!r || !r->table) return FA_OK;
  if (r->length < 0 || r->rot_dim < 0 || r->rot_dim > d || r->rot_dim % 16) return FA_ERR_RANGE;
  return aligned16(r->table) ? FA_OK : FA_ERR_ALIGN;
}

int check_kv(const fa_paged_kv* kv) {
  if (kv->d != 64 && kv->d != 128) return FA_ERR_HEAD_DIM;
  if (kv->num_pages < 0 || kv->Hkv < 0) return FA_ERR_SHAPE;
  const int ps = kv->page_size;
  if (ps <= 0 || !(ps % 128 == 0 || (ps < 128 && ps >= 8 && (ps & (ps - 1)) == 0))) return FA_ERR_RANGE;
  if (kv->num_pages == 0 || kv->Hkv == 0) return FA_OK;
  if (!kv->k || !kv->v) return FA_ERR_NULL;
  if (!aligned16(kv->k) || !aligned16(kv->v) || ((kv->page_stride | kv->head_stride | kv->token_stride) & 7))
    return FA_ERR_ALIGN;
  return FA_OK;
}

// sequences of a batch: the kernels' searches and shares round B up in 32 bits
constexpr int MAX_SEQUENCES = 1 << 30;

HeadsDev dev(const fa_heads* h) {
  return HeadsDev{static_cast<uint16_t*>(h->ptr), h->batch_stride, h->token_stride, h->head_stride, h->H};
}
RopeDev dev(const fa_rope* r) {
  if (!r || !r->table) return RopeDev{nullptr, 0, 0};
  return RopeDev{r->table, r->length, r->rot_dim};
}

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

// A kernel that waits on the device for the previous kernel of the stream (wait_previous_grid):
// its blocks may be set up while that one still runs.
template <typename... P, typename... A>
int launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return fa_host::launched(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// f(type, interleaved, full) for the eight instantiations of a kernel of head dimension d
template <typename F>
int by_type(fa_dtype dtype, const fa_rope* rope, int d, F f) {
  const bool full = rope && rope->table && rope->rot_dim == d;
  auto with_pairs = [&](auto bf, auto inter) {
    return full ? f(bf, inter, std::true_type{}) : f(bf, inter, std::false_type{});
  };
  auto with_type = [&](auto bf) {
    return rope && rope->interleaved ? with_pairs(bf, std::true_type{}) : with_pairs(bf, std::false_type{});
  };
  return dtype == FA_BF16 ? with_type(std::true_type{}) : with_type(std::false_type{});
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

// ------------------------------------------------------------------------- paged attention
// The kernel form for groups of G query heads and at most max_q new tokens: 0 = PAIR, else SPLIT
// with that many copies of each row, as many as fit into a tile of 128 rows (up to 4).
int paged_form(int G, int max_q) {
  const long long rows = (long long)G * max_q;
  return rows <= 32 ? 4 : rows <= 64 ? 2 : rows <= 128 ? 1 : 0;
}
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
size_t paged_records_bytes(int sms) { return round256((size_t)sms * 8 * sizeof(int)); }
size_t paged_parts_bytes(int sms, int d, int form) {
  return round256((size_t)sms * 2 * paged::part_floats(d, form == 0 ? 256 : 128 / form) * sizeof(float));
}

// A tensor of 16-bit rows of d elements with `dims - 1` outer axes; boxes of 64 columns, 128-byte
// swizzle. The stride of an axis of one element is never used; any valid one stands in for it.
int paged_map(CUtensorMap* m, const void* base, bool bf16, int dims, int d, std::initializer_list<uint64_t> size,
              std::initializer_list<long long> stride, std::initializer_list<uint32_t> box) {
  fa_host::EncodeTiledFn enc = fa_host::encode_tiled();
  if (!enc) return FA_ERR_TENSOR_MAP;
  cuuint64_t gd[4] = {(cuuint64_t)d}, gs[3];
  cuuint32_t bx[4] = {64}, es[4] = {1, 1, 1, 1};
  for (int i = 0; i < dims - 1; ++i) {
    gd[i + 1] = size.begin()[i];
    const long long s = stride.begin()[i];
    if (gd[i + 1] > 1 && s <= 0) return FA_ERR_TENSOR_MAP;
    gs[i] = gd[i + 1] > 1 ? (cuuint64_t)s * 2 : (cuuint64_t)d * 2;
    bx[i + 1] = box.begin()[i];
  }
  const CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims,
                         const_cast<void*>(base), gd, gs, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_TENSOR_MAP;
}

std::mutex g_attr_mu;

template <int D, bool BF16, bool SPLIT, int REP, bool DIRECT = true>
int launch_paged(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const paged::Params& p,
                 int index, int blocks, cudaStream_t st) {
  constexpr int SMEM = paged::Layout<D, SPLIT>::SMEM_BYTES, ROWS = SPLIT ? 128 / REP : 256;
  auto kern = paged::fa_paged_kernel<D, BF16, SPLIT, REP, DIRECT>;
  static bool attr_set[fa_host::MAX_DEVICES] = {};
  {
    std::lock_guard<std::mutex> lk(g_attr_mu);
    if (!attr_set[index]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
        return FA_ERR_CUDA;
      attr_set[index] = true;
    }
  }
  const int rc = launch_dependent(kern, dim3(blocks), dim3(paged::NUM_THREADS), SMEM, st, mq, mk, mv, p);
  if (rc != FA_OK || p.whole) return rc;
  // a warp joins 2 rows, or 1
  return launch_dependent(paged::fa_paged_combine_kernel<D, BF16, ROWS>, dim3(blocks, ROWS > 128 ? ROWS / 16 : ROWS / 8),
                          dim3(paged::COMBINE_THREADS), 0, st, p);
}

template <int D, bool BF16>
int paged_forms(int form, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                const paged::Params& p, int index, int blocks, cudaStream_t st) {
  switch (form) {
    case 4: return launch_paged<D, BF16, true, 4>(mq, mk, mv, p, index, blocks, st);
    case 2: return launch_paged<D, BF16, true, 2>(mq, mk, mv, p, index, blocks, st);
    case 1: return launch_paged<D, BF16, true, 1>(mq, mk, mv, p, index, blocks, st);
    default:
      return p.direct ? launch_paged<D, BF16, false, 1, true>(mq, mk, mv, p, index, blocks, st)
                      : launch_paged<D, BF16, false, 1, false>(mq, mk, mv, p, index, blocks, st);
  }
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
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (!kv || !q || !O) return FA_ERR_NULL;
  int rc = check_kv(kv);
  if (rc != FA_OK) return rc;
  if (B < 0 || T < 0 || table_stride < 0 || max_q < 1 || q->H < 0 || q->H != O->H) return FA_ERR_SHAPE;
  if (!(scale >= 0.f) || !isfinite(scale)) return FA_ERR_SCALE;
  if (B == 0 || T == 0 || q->H == 0) return FA_OK;
  if (kv->num_pages == 0 || kv->Hkv == 0 || q->H % kv->Hkv || q->H / kv->Hkv > 128 || B > MAX_SEQUENCES ||
      (long long)T * q->H > 0x7fffffffLL)
    return FA_ERR_SHAPE;
  if ((rc = check_heads(q)) != FA_OK || (rc = check_heads(O)) != FA_OK) return rc;
  if (!cu_seqlens || !seq_lens || (!block_table && table_stride)) return FA_ERR_NULL;
  if (!aligned4(cu_seqlens) || !aligned4(seq_lens) || !aligned4(block_table) || !aligned4(L)) return FA_ERR_ALIGN;
  if ((uintptr_t)workspace & 255) return FA_ERR_ALIGN;
  int index = 0, sms = 0;
  if ((rc = fa_host::current_device(&index, &sms)) != FA_OK) return rc;
  const int G = q->H / kv->Hkv, form = paged_form(G, max_q);
  const bool whole = (long long)table_stride * kv->page_size <= paged::WHOLE_TILES * paged::BN;
  if (!whole && (!workspace || workspace_bytes < paged_records_bytes(sms) + paged_parts_bytes(sms, kv->d, form)))
    return FA_ERR_WORKSPACE;
  paged::Params p = {};
  if ((rc = fa_host::status_word(&p.status)) != FA_OK) return rc;
  p.o = dev(O);
  p.L = L;
  p.num_pages = kv->num_pages;
  p.page_size = kv->page_size;
  p.box_keys = kv->page_size < 128 ? kv->page_size : 128;
  p.Hkv = kv->Hkv;
  p.G = G;
  p.by_g = (65536u + G - 1) / G;
  p.tpt = (form == 0 ? 128 : 128 / form) / G;
  p.cu = cu_seqlens;
  p.lens = seq_lens;
  p.table = block_table;
  p.table_stride = table_stride;
  p.B = B;
  p.T = T;
  const long long cap = (long long)table_stride * kv->page_size;
  p.cap = cap < 0x7fffff00LL ? (int)cap : 0x7fffff00;
  p.causal = causal != 0;
  p.c = scale * 1.4426950408889634f;
  p.wait_limit_ns = fa_host::wait_limit_ns();
  p.whole = whole;
  // without units: whole items that fit the SMs at once, or one sequence whose key heads share nine
  // tenths of them (8 heads over 1001 keys: 9.5 us against 12.0 by units, 28 over 8001, 140 SMs, 26.2
  // against 27.5). With fewer SMs in use it may cost more, 80 heads over 8001 keys 64.7 against 58.2 us,
  // or less: 27 heads, 135 SMs, 25.7 against 27.3, and over 1001 keys 10.5 against 12.5.
  const long long heads = (long long)B * kv->Hkv;
  if (whole) {
    const int per_item = p.tpt * (form == 0 ? 2 : 1);
    const long long parts = max_q <= per_item ? 1 : (max_q - 1) / per_item + 1;  // blocks of tokens
    if (heads * parts <= sms) p.direct = (int)parts;
  } else if (form != 0 && B == 1 && kv->Hkv <= sms && sms / kv->Hkv * kv->Hkv * 10 >= sms * 9) {
    p.direct = sms / kv->Hkv;
  }
  const int blocks = p.direct ? (int)heads * p.direct : sms;
  if (!whole) {
    p.records = static_cast<int*>(workspace);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + paged_records_bytes(sms));
    p.parts_len = (long long)((workspace_bytes - paged_records_bytes(sms)) / sizeof(float));
    const long long most = fa_host::debug_part_cap();
    if (most >= 0 && most < p.parts_len) p.parts_len = most;
  }
  const bool bf16 = dtype == FA_BF16;
  CUtensorMap mq, mk, mv;
  // Q as [T, Hq, d]: a box is 64 columns of the G heads of a key head for tpt tokens
  if ((rc = paged_map(&mq, q->ptr, bf16, 3, kv->d, {(uint64_t)q->H, (uint64_t)T}, {q->head_stride, q->token_stride},
                      {(uint32_t)G, (uint32_t)p.tpt})) != FA_OK)
    return rc;
  for (int i = 0; i < 2; ++i)
    if ((rc = paged_map(i ? &mv : &mk, i ? kv->v : kv->k, bf16, 4, kv->d,
                        {(uint64_t)kv->page_size, (uint64_t)kv->Hkv, (uint64_t)kv->num_pages},
                        {kv->token_stride, kv->head_stride, kv->page_stride}, {(uint32_t)p.box_keys, 1, 1})) != FA_OK)
      return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (kv->d == 64) return bf16 ? paged_forms<64, true>(form, mq, mk, mv, p, index, blocks, st) : paged_forms<64, false>(form, mq, mk, mv, p, index, blocks, st);
  return bf16 ? paged_forms<128, true>(form, mq, mk, mv, p, index, blocks, st) : paged_forms<128, false>(form, mq, mk, mv, p, index, blocks, st);
}

}  // extern "C"
