// fa_decoder_host.h -- what the translation units behind include/fa_decoder.h share on the host: checks
// of arguments, launches, and the call of attention over a paged cache. Internal; not part of the C ABI.
#pragma once
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

// hidden: two copies of the library in one process (the range-checked build beside the release build) each
// keep their own launch_paged<>::attr_set, which would else be one symbol for the whole process
namespace fa_decoder __attribute__((visibility("hidden"))) {

using namespace fa;

inline bool aligned16(const void* ptr) { return ((uintptr_t)ptr & 15) == 0; }
inline bool aligned4(const void* ptr) { return ((uintptr_t)ptr & 3) == 0; }

// Checks of one set of rows; a set with H == 0 passes.
inline int check_heads(const fa_heads* h) {
  if (h->H < 0) return FA_ERR_SHAPE;
  if (h->H == 0) return FA_OK;
  if (!h->ptr) return FA_ERR_NULL;
  if (!aligned16(h->ptr) || ((h->batch_stride | h->token_stride | h->head_stride) & 7)) return FA_ERR_ALIGN;
  return FA_OK;
}

inline int check_rope(const fa_rope* r, int d) {
  if (!r || !r->table) return FA_OK;
  if (r->length < 0 || r->rot_dim < 0 || r->rot_dim > d || r->rot_dim % 16) return FA_ERR_RANGE;
  return aligned16(r->table) ? FA_OK : FA_ERR_ALIGN;
}

// `unit`: its strides are multiples of that many elements (16 bytes)
inline int check_kv(const fa_paged_kv* kv, int unit = 8) {
  if (kv->d != 64 && kv->d != 128) return FA_ERR_HEAD_DIM;
  if (kv->num_pages < 0 || kv->Hkv < 0) return FA_ERR_SHAPE;
  const int ps = kv->page_size;
  if (ps <= 0 || !(ps % 128 == 0 || (ps < 128 && ps >= 8 && (ps & (ps - 1)) == 0))) return FA_ERR_RANGE;
  if (kv->num_pages == 0 || kv->Hkv == 0) return FA_OK;
  if (!kv->k || !kv->v) return FA_ERR_NULL;
  if (!aligned16(kv->k) || !aligned16(kv->v) || ((kv->page_stride | kv->head_stride | kv->token_stride) & (unit - 1)))
    return FA_ERR_ALIGN;
  return FA_OK;
}

// sequences of a batch: the kernels' searches and shares round B up in 32 bits
constexpr int MAX_SEQUENCES = 1 << 30;

inline HeadsDev dev(const fa_heads* h) {
  return HeadsDev{static_cast<uint16_t*>(h->ptr), h->batch_stride, h->token_stride, h->head_stride, h->H};
}
inline RopeDev dev(const fa_rope* r) {
  if (!r || !r->table) return RopeDev{nullptr, 0, 0};
  return RopeDev{r->table, r->length, r->rot_dim};
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

// ------------------------------------------------------------------------- paged attention
// The kernel form for groups of G query heads and at most max_q new tokens: 0 = PAIR, else SPLIT
// with that many copies of each row, as many as fit into a tile of 128 rows (up to 4).
inline int paged_form(int G, int max_q) {
  const long long rows = (long long)G * max_q;
  return rows <= 32 ? 4 : rows <= 64 ? 2 : rows <= 128 ? 1 : 0;
}
inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
inline size_t paged_records_bytes(int sms) { return round256((size_t)sms * 8 * sizeof(int)); }
inline size_t paged_parts_bytes(int sms, int d, int form) {
  return round256((size_t)sms * 2 * paged::part_floats(d, form == 0 ? 256 : 128 / form) * sizeof(float));
}

// A tensor of rows of d elements with `dims - 1` outer axes: 16-bit ones in boxes of 64 columns, 128-byte
// swizzle, 8-bit ones in boxes of whole rows, as they lie or swizzled as K-major operands are. The stride of an axis of one element is never used; any valid one stands in for it.
enum RowKind { ROWS16, ROWS8, ROWS8_SWIZZLED };
inline int paged_map(CUtensorMap* m, const void* base, bool bf16, int dims, int d, std::initializer_list<uint64_t> size,
                     std::initializer_list<long long> stride, std::initializer_list<uint32_t> box, RowKind kind = ROWS16) {
  fa_host::EncodeTiledFn enc = fa_host::encode_tiled();
  if (!enc) return FA_ERR_TENSOR_MAP;
  cuuint64_t gd[4] = {(cuuint64_t)d}, gs[3];
  const bool wide = kind == ROWS16;
  const int elem_bytes = wide ? 2 : 1;
  const CUtensorMapSwizzle swizzle = kind == ROWS8 ? CU_TENSOR_MAP_SWIZZLE_NONE
                                     : !wide && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  cuuint32_t bx[4] = {wide ? 64u : (cuuint32_t)d}, es[4] = {1, 1, 1, 1};
  for (int i = 0; i < dims - 1; ++i) {
    gd[i + 1] = size.begin()[i];
    const long long s = stride.begin()[i];
    if (gd[i + 1] > 1 && s <= 0) return FA_ERR_TENSOR_MAP;
    gs[i] = gd[i + 1] > 1 ? (cuuint64_t)s * elem_bytes : (cuuint64_t)d * elem_bytes;
    bx[i + 1] = box.begin()[i];
  }
  const CUresult r = enc(m, !wide ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims,
                         const_cast<void*>(base), gd, gs, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_TENSOR_MAP;
}

inline std::mutex g_attr_mu;

template <int D, bool BF16, bool SPLIT, int REP, bool F8, bool DIRECT = true>
int launch_paged(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const paged::Params& p,
                 int index, int blocks, cudaStream_t st) {
  constexpr int SMEM = paged::Layout<D, SPLIT, F8 ? (BF16 ? 2 : 3) : 0>::SMEM_BYTES, ROWS = SPLIT ? 128 / REP : 256;
  auto kern = paged::fa_paged_kernel<D, BF16, SPLIT, REP, DIRECT, F8>;
  static bool attr_set[fa_host::MAX_DEVICES] = {};
  {
    std::lock_guard<std::mutex> lk(g_attr_mu);
    if (!attr_set[index]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
        return FA_ERR_CUDA;
      attr_set[index] = true;
    }
  }
  const int rc = launch_dependent(kern, dim3(blocks), dim3(paged::num_warps(F8) * 32), SMEM, st, mq, mk, mv, p);
  if (rc != FA_OK || p.whole) return rc;
  // a warp joins 2 rows, or 1
  return launch_dependent(paged::fa_paged_combine_kernel<D, BF16, ROWS>, dim3(blocks, ROWS > 128 ? ROWS / 16 : ROWS / 8),
                          dim3(paged::COMBINE_THREADS), 0, st, p);
}

// Rows of a tile of fa_rows8.cuh for groups of G query heads and at most max_q new tokens, 0: more than it takes. (More
// rows take its threads too long: 32 rows of 64 ragged sequences, d 128, 320 us against 161 in fa_paged.cuh.)
inline int rows8_of(int G, int max_q) { return (long long)G * max_q <= 8 ? 8 : (long long)G * max_q <= 16 ? 16 : 0; }

// The launch of fa_rows8.cuh's kernels (fa_rows8.cu).
__attribute__((visibility("hidden"))) int launch_rows8(int d, bool bf16, const CUtensorMap& mk, const CUtensorMap& mv,
                                                       const paged::Params& p, int index, int blocks, cudaStream_t st);

template <int D, bool BF16, bool F8>
int paged_forms(int form, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                const paged::Params& p, int index, int blocks, cudaStream_t st) {
  switch (form) {
    case 4:
      if (F8 && p.rows8) return launch_rows8(D, BF16, mk, mv, p, index, blocks, st);
      return launch_paged<D, BF16, true, 4, F8>(mq, mk, mv, p, index, blocks, st);
    case 2: return launch_paged<D, BF16, true, 2, F8>(mq, mk, mv, p, index, blocks, st);
    case 1: return launch_paged<D, BF16, true, 1, F8>(mq, mk, mv, p, index, blocks, st);
    default:
      return p.direct ? launch_paged<D, BF16, false, 1, F8, true>(mq, mk, mv, p, index, blocks, st)
                      : launch_paged<D, BF16, false, 1, F8, false>(mq, mk, mv, p, index, blocks, st);
  }
}

// fa_fwd_paged, and with F8 (scales k_scale, v_scale) fa_fwd_paged_fp8
template <bool F8>
int attend_paged(const fa_paged_kv* kv, const float* k_scale, const float* v_scale, const fa_heads* q,
                 const fa_heads* O, float* L, int B, int T, int max_q, const int* cu_seqlens, const int* seq_lens,
                 const int* block_table, int table_stride, float scale, int causal, fa_dtype dtype, void* workspace,
                 size_t workspace_bytes, void* stream) {
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (!kv || !q || !O) return FA_ERR_NULL;
  int rc = check_kv(kv, F8 ? 16 : 8);
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
  if (F8 && (!k_scale || !v_scale)) return FA_ERR_NULL;
  if (F8 && (!aligned4(k_scale) || !aligned4(v_scale))) return FA_ERR_ALIGN;
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
  p.page_shift = -1;
  for (int x = 0; x < 31; ++x)
    if (kv->page_size == 1 << x) p.page_shift = x;
  p.box_keys = kv->page_size < 128 ? kv->page_size : 128;
  p.Hkv = kv->Hkv;
  p.G = G;
  p.by_g = (65536u + G - 1) / G;
  p.tpt = (form == 0 ? 128 : 128 / form) / G;
  if (F8 && (p.rows8 = rows8_of(G, max_q)) != 0) p.tpt = p.rows8 / G;
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
  p.ks = k_scale;
  p.vs = v_scale;
  if (F8) p.q = dev(q);
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
  CUtensorMap mq = {}, mk, mv;
  // Q as [T, Hq, d]: a box is 64 columns of the G heads of a key head for tpt tokens
  if (!F8 && (rc = paged_map(&mq, q->ptr, bf16, 3, kv->d, {(uint64_t)q->H, (uint64_t)T}, {q->head_stride, q->token_stride},
                      {(uint32_t)G, (uint32_t)p.tpt})) != FA_OK)
    return rc;
  for (int i = 0; i < 2; ++i)
    if ((rc = paged_map(i ? &mv : &mk, i ? kv->v : kv->k, bf16, 4, kv->d,
                        {(uint64_t)kv->page_size, (uint64_t)kv->Hkv, (uint64_t)kv->num_pages},
                        {kv->token_stride, kv->head_stride, kv->page_stride}, {(uint32_t)p.box_keys, 1, 1},
                        !F8 ? ROWS16 : i && !p.rows8 ? ROWS8 : ROWS8_SWIZZLED)) != FA_OK)
      return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (kv->d == 64) return bf16 ? paged_forms<64, true, F8>(form, mq, mk, mv, p, index, blocks, st) : paged_forms<64, false, F8>(form, mq, mk, mv, p, index, blocks, st);
  return bf16 ? paged_forms<128, true, F8>(form, mq, mk, mv, p, index, blocks, st) : paged_forms<128, false, F8>(form, mq, mk, mv, p, index, blocks, st);
}

}  // namespace fa_decoder
