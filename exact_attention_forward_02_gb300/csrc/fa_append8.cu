// fa_append8.cu -- the C ABI of include/fa_decoder.h, part: the append to a cache held in 8 bits. The kernel
// lives in fa_append8.cuh.
#include "fa_append8.cuh"
#include "fa_decoder_host.h"

namespace {

using namespace fa;
using namespace fa_decoder;

// Warps of a unit: as many as hold the rows that a page may get in their lanes, 4 rows of a lane (4 blocks of an
// SM; with 8 rows, 2 blocks, 29582 ragged tokens of 8 heads, d 128, took 72 us for 56) or for large pages 8.
template <int D, bool BF16, bool INTER, bool FULL>
int launch_append8(const Append8Params& p, cudaStream_t st) {
  constexpr int LANES = 256 / D;  // rows of a warp
  const int rows = p.page_size < p.T ? p.page_size : p.T;
  auto go = [&](auto w, auto r) {
    constexpr int W = decltype(w)::value, ROWS = decltype(r)::value, UNITS = ROW_WARPS / W;
    const long long blocks = (p.units + UNITS - 1) / UNITS + 1;  // the last one looks over cu_seqlens
    if (blocks > 0x7fffffffLL) return (int)FA_ERR_SHAPE;
    return launch_dependent(fa_paged_append8_kernel<D, BF16, INTER, FULL, W, ROWS>, dim3((unsigned)blocks), dim3(ROW_THREADS),
                            0, st, p);
  };
  using std::integral_constant;
  if (rows <= 8 * LANES) return go(integral_constant<int, 1>{}, integral_constant<int, 8>{});
  if (rows <= 16 * LANES) return go(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  if (rows <= 32 * LANES) return go(integral_constant<int, 8>{}, integral_constant<int, 4>{});
  return go(integral_constant<int, 8>{}, integral_constant<int, 8>{});
}

}  // namespace

extern "C" {

int fa_paged_append_fp8(const fa_paged_kv* kv, float* k_scale, float* v_scale, const fa_heads* k, const fa_heads* v,
                        int B, int T, const int* cu_seqlens, const int* seq_lens, const int* block_table,
                        int table_stride, const fa_rope* rope, fa_dtype dtype, void* stream) {
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (!kv || !k || !v) return FA_ERR_NULL;
  int rc = check_kv(kv, 16);
  if (rc != FA_OK) return rc;
  if (B < 0 || T < 0 || table_stride < 0 || k->H != kv->Hkv || v->H != kv->Hkv) return FA_ERR_SHAPE;
  if ((rc = check_rope(rope, kv->d)) != FA_OK) return rc;
  if (B == 0 || T == 0 || kv->Hkv == 0) return FA_OK;
  if ((long long)T * 2 * kv->Hkv > 0x7fffffffLL || B > MAX_SEQUENCES) return FA_ERR_SHAPE;
  if ((rc = check_heads(k)) != FA_OK || (rc = check_heads(v)) != FA_OK) return rc;
  if (!cu_seqlens || !seq_lens || (!block_table && table_stride)) return FA_ERR_NULL;
  if (kv->num_pages && (!k_scale || !v_scale)) return FA_ERR_NULL;
  if (!aligned4(cu_seqlens) || !aligned4(seq_lens) || !aligned4(block_table) || !aligned4(k_scale) ||
      !aligned4(v_scale))
    return FA_ERR_ALIGN;
  int index = 0, sms = 0;
  if ((rc = fa_host::current_device(&index, &sms)) != FA_OK) return rc;
  Append8Params p = {};
  if ((rc = fa_host::status_word(&p.status)) != FA_OK) return rc;
  p.k = dev(k);
  p.v = dev(v);
  p.kp = static_cast<uint8_t*>(kv->k);
  p.vp = static_cast<uint8_t*>(kv->v);
  p.ks = k_scale;
  p.vs = v_scale;
  p.page_stride = kv->page_stride;
  p.head_stride = kv->head_stride;
  p.token_stride = kv->token_stride;
  p.num_pages = kv->num_pages;
  p.page_size = kv->page_size;
  p.Hkv = kv->Hkv;
  p.cu = cu_seqlens;
  p.lens = seq_lens;
  p.table = block_table;
  p.table_stride = table_stride;
  p.B = B;
  p.T = T;
  p.units = ((long long)T / kv->page_size + 2LL * B) * 2 * kv->Hkv;
  p.rope = dev(rope);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return by_type(dtype, rope, kv->d, [&](auto bf, auto inter, auto full) {
    return kv->d == 64 ? launch_append8<64, bf, inter, full>(p, st) : launch_append8<128, bf, inter, full>(p, st);
  });
}

}  // extern "C"
