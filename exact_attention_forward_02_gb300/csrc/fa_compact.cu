// fa_compact.cu -- the C ABI of include/fa_decoder.h, part: attention over a cache held in 8 bits. The kernels live
// in fa_paged.cuh (chunks) and fa_rows8.cuh (single tokens and drafts).
#include "fa_decoder_host.h"

using namespace fa_decoder;

extern "C" {

int fa_fwd_paged_fp8(const fa_paged_kv* kv, const float* k_scale, const float* v_scale, const fa_heads* q,
                     const fa_heads* O, float* L, int B, int T, int max_q, const int* cu_seqlens, const int* seq_lens,
                     const int* block_table, int table_stride, float scale, int causal, fa_dtype dtype,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return attend_paged<true>(kv, k_scale, v_scale, q, O, L, B, T, max_q, cu_seqlens, seq_lens, block_table,
                            table_stride, scale, causal, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
