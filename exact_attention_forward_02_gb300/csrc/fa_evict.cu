// fa_evict.cu -- the C ABI of include/fa_decoder.h, part: weights of cached tokens, and their eviction. The
// kernels live in fa_weigh.cuh and fa_evict.cuh.
#include "fa_decoder_host.h"
#include "fa_evict.cuh"
#include "fa_weigh.cuh"

namespace {

using namespace fa;
using namespace fa_decoder;

// once per kernel and device: more than 48 KB of shared memory
int allow_smem(const void* kernel, int bytes, bool* done) {
  std::lock_guard<std::mutex> lk(g_attr_mu);
  if (!*done) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return FA_ERR_CUDA;
    *done = true;
  }
  return FA_OK;
}

template <int D, bool BF16, int MODE>
int launch_weigh(const CUtensorMap& mq, const CUtensorMap& mk, const weigh::Params& p, int index, int sms,
                 cudaStream_t st) {
  constexpr int SMEM = weigh::Layout<D, BF16, MODE>::SMEM_BYTES;
  auto kern = weigh::fa_weigh_kernel<D, BF16, MODE>;
  static bool done[fa_host::MAX_DEVICES] = {};
  const int rc = allow_smem(reinterpret_cast<const void*>(kern), SMEM, &done[index]);
  if (rc != FA_OK) return rc;
  return launch_dependent(kern, dim3(sms), dim3(weigh::num_warps(MODE) * 32), SMEM, st, mq, mk, p);
}

size_t evict_list_bytes(int B, int Hkv, int budget) { return round256((size_t)B * Hkv * budget * sizeof(int2)); }
size_t evict_first_bytes(int B, int Hkv) { return round256((size_t)B * Hkv * sizeof(int)); }

template <bool F8>
int launch_evict(evict::Params& p, int index, cudaStream_t st) {
  const long long heads = (long long)p.B * p.Hkv;
  auto select = evict::fa_evict_select_kernel<F8>;
  const int least = F8 ? 2 * evict::SCALE_PAGES : 0;
  static bool done[fa_host::MAX_DEVICES] = {};
  const int rc = allow_smem(reinterpret_cast<const void*>(select), (int)sizeof(evict::SelectSmem) + evict::KEY_CAP * 4,
                            &done[index]);
  if (rc != FA_OK) return rc;
  p.keys = p.cap < evict::KEY_CAP ? p.cap : evict::KEY_CAP;
  const size_t smem = sizeof(evict::SelectSmem) + (size_t)(p.keys > least ? p.keys : least) * 4;
  const int rc1 = launch_dependent(select, dim3((unsigned)heads), dim3(evict::SELECT_THREADS), smem, st, p);
  if (rc1 != FA_OK) return rc1;
  return launch_dependent(evict::fa_evict_move_kernel<F8>, dim3((unsigned)(heads * (2 * p.slices + 1))),
                          dim3(evict::MOVE_THREADS), 0, st, p);
}

}  // namespace

extern "C" {

int fa_paged_key_weights(const fa_paged_kv* kv, const float* k_scale, const fa_heads* q, const float* L, float* weights,
                         int B, int T, int max_q, const int* cu_seqlens, const int* seq_lens, const int* block_table,
                         int table_stride, float scale, int causal, fa_dtype dtype, void* stream) {
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (!kv || !q) return FA_ERR_NULL;
  const bool f8 = k_scale != nullptr;
  fa_paged_kv keys = *kv;  // V is not looked at
  keys.v = keys.k;
  int rc = check_kv(&keys, f8 ? 16 : 8);
  if (rc != FA_OK) return rc;
  if (B < 0 || T < 0 || table_stride < 0 || max_q < 1 || q->H < 0) return FA_ERR_SHAPE;
  if (!(scale >= 0.f) || !isfinite(scale)) return FA_ERR_SCALE;
  if (B == 0 || T == 0 || q->H == 0) return FA_OK;
  if (kv->num_pages == 0 || kv->Hkv == 0 || q->H % kv->Hkv || q->H / kv->Hkv > 128 || B > MAX_SEQUENCES ||
      (long long)T * q->H > 0x7fffffffLL || (long long)kv->Hkv * kv->page_size > 0xffffffffLL)
    return FA_ERR_SHAPE;
  if ((rc = check_heads(q)) != FA_OK) return rc;
  if (!L || !weights || !cu_seqlens || !seq_lens || (!block_table && table_stride)) return FA_ERR_NULL;
  if (!aligned4(cu_seqlens) || !aligned4(seq_lens) || !aligned4(block_table) || !aligned4(L) || !aligned4(weights) ||
      !aligned4(k_scale))
    return FA_ERR_ALIGN;
  int index = 0, sms = 0;
  if ((rc = fa_host::current_device(&index, &sms)) != FA_OK) return rc;
  weigh::Params p = {};
  if ((rc = fa_host::status_word(&p.status)) != FA_OK) return rc;
  p.L = L;
  p.ks = k_scale;
  p.w = weights;
  p.num_pages = kv->num_pages;
  p.page_size = kv->page_size;
  p.box_keys = kv->page_size < 128 ? kv->page_size : 128;
  p.Hkv = kv->Hkv;
  p.Hq = q->H;
  p.G = q->H / kv->Hkv;
  p.by_g = (65536u + p.G - 1) / p.G;
  // a tile of rows holds the most new tokens that a sequence has, or as many as make 128 rows
  p.tpt = 128 / p.G < max_q ? 128 / p.G : max_q;
  p.cols = p.tpt * p.G;
  p.cu = cu_seqlens;
  p.lens = seq_lens;
  p.table = block_table;
  p.table_stride = table_stride;
  p.B = B;
  p.T = T;
  p.causal = causal != 0;
  const long long cap = (long long)table_stride * kv->page_size;
  p.cap = cap < 0x7fffff00LL ? (int)cap : 0x7fffff00;
  p.c = scale * 1.4426950408889634f;
  p.wait_limit_ns = fa_host::wait_limit_ns();
  const bool bf16 = dtype == FA_BF16, held = f8 && p.cols <= weigh::HELD_ROWS;
  p.page_shift = -1;
  for (int x = 0; x < 31; ++x)
    if (kv->page_size == 1 << x) p.page_shift = x;
  if (held) p.q = dev(q);
  CUtensorMap mq = {}, mk;
  if (!held && (rc = paged_map(&mq, q->ptr, bf16, 3, kv->d, {(uint64_t)q->H, (uint64_t)T}, {q->head_stride, q->token_stride},
                      {(uint32_t)p.G, (uint32_t)p.tpt})) != FA_OK)
    return rc;
  if ((rc = paged_map(&mk, kv->k, bf16, 4, kv->d, {(uint64_t)kv->page_size, (uint64_t)kv->Hkv, (uint64_t)kv->num_pages},
                      {kv->token_stride, kv->head_stride, kv->page_stride}, {(uint32_t)p.box_keys, 1, 1},
                      held ? ROWS8_SWIZZLED : f8 ? ROWS8 : ROWS16)) != FA_OK)
    return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto m) {
    constexpr int M = decltype(m)::value;
    if (kv->d == 64)
      return bf16 ? launch_weigh<64, true, M>(mq, mk, p, index, sms, st) : launch_weigh<64, false, M>(mq, mk, p, index, sms, st);
    return bf16 ? launch_weigh<128, true, M>(mq, mk, p, index, sms, st) : launch_weigh<128, false, M>(mq, mk, p, index, sms, st);
  };
  if (held) return go(std::integral_constant<int, weigh::HELD>{});
  return f8 ? go(std::integral_constant<int, weigh::TURNED>{}) : go(std::integral_constant<int, weigh::HALF>{});
}

size_t fa_paged_evict_workspace_bytes(int B, int Hkv, int budget, int held8) {
  if (B <= 0 || Hkv <= 0 || budget <= 0) return 0;
  const size_t ratio = held8 ? round256((size_t)2 * B * Hkv * budget * sizeof(float)) : 0;
  return evict_list_bytes(B, Hkv, budget) + evict_first_bytes(B, Hkv) + ratio;
}

int fa_paged_evict(const fa_paged_kv* kv, float* k_scale, float* v_scale, float* weights, int B, const int* seq_lens,
                   const int* block_table, int table_stride, int budget, int recent, int* kept, int* new_lens,
                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!kv) return FA_ERR_NULL;
  if (!k_scale != !v_scale) return FA_ERR_NULL;
  const bool f8 = k_scale != nullptr;
  int rc = check_kv(kv, f8 ? 16 : 8);
  if (rc != FA_OK) return rc;
  if (B < 0 || table_stride < 0 || budget < 1 || recent < 0 || recent > budget) return FA_ERR_SHAPE;
  if (B == 0 || kv->Hkv == 0) return FA_OK;
  // (a budget that leaves the kernels' strides over it room in 32 bits)
  if (B > MAX_SEQUENCES || (long long)B * kv->Hkv > 0x1ffffff || budget > 0x7fff0000) return FA_ERR_SHAPE;
  if (!seq_lens || !kept || !new_lens || (!block_table && table_stride) || (kv->num_pages && !weights)) return FA_ERR_NULL;
  if (!aligned4(seq_lens) || !aligned4(block_table) || !aligned4(kept) || !aligned4(new_lens) || !aligned4(weights) ||
      !aligned4(k_scale) || !aligned4(v_scale) || ((uintptr_t)workspace & 255))
    return FA_ERR_ALIGN;
  if (!workspace || workspace_bytes < fa_paged_evict_workspace_bytes(B, kv->Hkv, budget, f8)) return FA_ERR_WORKSPACE;
  int index = 0, sms = 0;
  if ((rc = fa_host::current_device(&index, &sms)) != FA_OK) return rc;
  evict::Params p = {};
  if ((rc = fa_host::status_word(&p.status)) != FA_OK) return rc;
  const int elem = f8 ? 1 : 2;
  p.pages[0] = static_cast<uint8_t*>(kv->k);
  p.pages[1] = static_cast<uint8_t*>(kv->v);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.w = weights;
  p.page_bytes = kv->page_stride * elem;
  p.head_bytes = kv->head_stride * elem;
  p.token_bytes = kv->token_stride * elem;
  p.num_pages = kv->num_pages;
  p.page_size = kv->page_size;
  p.page_shift = -1;
  for (int x = 0; x < 31; ++x)
    if (kv->page_size == 1 << x) p.page_shift = x;
  p.Hkv = kv->Hkv;
  p.lens = seq_lens;
  p.table = block_table;
  p.table_stride = table_stride;
  p.B = B;
  // (and a length that leaves them room: a block's steps over its positions are up to 1024 wide)
  const long long cap = (long long)table_stride * kv->page_size;
  p.cap = cap < 0x7fff0000LL ? (int)cap : 0x7fff0000;
  p.budget = budget;
  p.recent = recent;
  p.kept = kept;
  p.new_lens = new_lens;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.src = reinterpret_cast<int2*>(ws);
  p.first = reinterpret_cast<int*>(ws + evict_list_bytes(B, kv->Hkv, budget));
  p.ratio = reinterpret_cast<float*>(ws + evict_list_bytes(B, kv->Hkv, budget) + evict_first_bytes(B, kv->Hkv));
  // whole rows where there are heads enough, else down to 32 bytes of them, so that the SMs have two blocks each
  p.row_pieces = kv->d * elem / 16;
  p.slice_pieces = p.row_pieces;
  while (p.slice_pieces > 2 && (long long)B * kv->Hkv * 2 * (p.row_pieces / p.slice_pieces) < 2LL * sms) p.slice_pieces /= 2;
  p.slices = p.row_pieces / p.slice_pieces;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return f8 ? launch_evict<true>(p, index, st) : launch_evict<false>(p, index, st);
}

}  // extern "C"
