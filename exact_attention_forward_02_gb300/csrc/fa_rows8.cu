// fa_rows8.cu -- launches of fa_rows8.cuh's kernels, for fa_fwd_paged_fp8.
#include "fa_decoder_host.h"
#include "fa_rows8.cuh"

namespace {

using namespace fa;
using namespace fa_decoder;

template <int D, bool BF16, int R>
int launch(const CUtensorMap& mk, const CUtensorMap& mv, const paged::Params& p, int index, int blocks,
                 cudaStream_t st) {
  constexpr int SMEM = paged::Layout8<D, BF16 ? 2 : 3, R>::SMEM_BYTES, ROWS = 32;
  auto kern = paged::fa_paged_rows8_kernel<D, BF16, R>;
  static bool attr_set[fa_host::MAX_DEVICES] = {};
  {
    std::lock_guard<std::mutex> lk(g_attr_mu);
    if (!attr_set[index]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
        return FA_ERR_CUDA;
      attr_set[index] = true;
    }
  }
  const int rc = launch_dependent(kern, dim3(blocks), dim3(paged::R8_THREADS), SMEM, st, mk, mv, p);
  if (rc != FA_OK || p.whole) return rc;
  return launch_dependent(paged::fa_paged_combine_kernel<D, BF16, ROWS>, dim3(blocks, R / 8),
                          dim3(paged::COMBINE_THREADS), 0, st, p);
}

template <int D, bool BF16>
int by_rows(const CUtensorMap& mk, const CUtensorMap& mv, const paged::Params& p, int index, int blocks,
            cudaStream_t st) {
  if (p.rows8 == 8) return launch<D, BF16, 8>(mk, mv, p, index, blocks, st);
  return launch<D, BF16, 16>(mk, mv, p, index, blocks, st);
}

}  // namespace

int fa_decoder::launch_rows8(int d, bool bf16, const CUtensorMap& mk, const CUtensorMap& mv, const paged::Params& p,
                             int index, int blocks, cudaStream_t st) {
  if (d == 64) return bf16 ? by_rows<64, true>(mk, mv, p, index, blocks, st) : by_rows<64, false>(mk, mv, p, index, blocks, st);
  return bf16 ? by_rows<128, true>(mk, mv, p, index, blocks, st) : by_rows<128, false>(mk, mv, p, index, blocks, st);
}
