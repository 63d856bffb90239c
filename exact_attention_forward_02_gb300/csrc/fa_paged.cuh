// fa_paged.cuh -- attention over a paged cache. Included by fa_decoder.cu.
#pragma once

#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include "fa_rope.cuh"

namespace fa {

struct PagedParams {
  HeadsDev q, o;
  float* L;
  const uint16_t *kp, *vp;
  long long page_stride, head_stride, token_stride;
  int num_pages, page_size, Hkv, G;
  const int *cu, *lens, *table;
  int table_stride, B, T;
  float c;
  int causal;
  int* status;
};

// One warp per (token row, query head), one key after another.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) fa_paged_simple_kernel(const __grid_constant__ PagedParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, Hq = p.Hkv * p.G;
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(unit / Hq), h = (int)(unit % Hq);
  if (t >= p.T) return;
  const int b = find_sequence(p.cu, p.B, t, lane);
  if (b < 0) return;
  int len = p.lens[b];
  const int pos = len - (p.cu[b + 1] - t);
  if (len > (long long)p.table_stride * p.page_size) {
    len = p.table_stride * p.page_size;
    if (lane == 0) atomicCAS(p.status, 0, FA_ERR_RANGE);
  }
  const int n = p.causal ? min(pos + 1, len) : len;
  auto load = [&](const uint16_t* src, float (&x)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 2) unpack2<BF16>(*reinterpret_cast<const uint32_t*>(src + lane * E + e), x[e], x[e + 1]);
  };
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  load(p.q.ptr + t * p.q.ts + h * p.q.hs, q);
  for (int j = 0; j < n; ++j) {
    const int page = p.table[(size_t)b * p.table_stride + j / p.page_size];
    float k[E] = {}, v[E] = {};
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicCAS(p.status, 0, FA_ERR_RANGE);
    } else {
      const long long at = page * p.page_stride + (h / p.G) * p.head_stride + (j % p.page_size) * p.token_stride;
      load(p.kp + at, k);
      load(p.vp + at, v);
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    s = row_sum<32>(s) * p.c;
    const float mn = fmaxf(m, s), a = ex2_approx(m - mn), w = ex2_approx(s - mn);
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * v[e];
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(p.o.ptr + t * p.o.ts + h * p.o.hs + lane * E + e) = pack2<BF16>(o[e] * inv, o[e + 1] * inv);
  if (p.L && lane == 0) p.L[(size_t)t * Hq + h] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace fa
