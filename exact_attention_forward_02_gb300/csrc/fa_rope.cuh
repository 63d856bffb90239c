// fa_rope.cuh -- per-row kernels over query, key and value heads: RMS norm + position rotation
// (forward and backward) and the append to a paged cache. Included by fa_decoder.cu.
//
// All of them read and write each row of d 16-bit elements once and are bound by HBM. A row is
// held by d/8 lanes, 8 elements (16 bytes) each, so that a warp has 2 (d = 128) or 4 (d = 64)
// rows in flight per load; a warp works on ONE token, so that its lanes load their angles of the
// rotation table once and keep them in registers over that token's heads.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "fa_decoder.h"
#include "sm103_ptx.cuh"

namespace fa {

struct HeadsDev {
  uint16_t* ptr;
  long long bs, ts, hs;  // batch, token and head stride in elements
  int H;
};
struct RopeDev {
  const float* table;
  int length, rot;  // rot = 0: no rotation
};

constexpr int ROW_THREADS = 256;
constexpr int ROW_WARPS = ROW_THREADS / 32;
constexpr int ROW_UNROLL = 4;          // rows of one lane group loaded before the first is used
constexpr int ROW_BWD_MAX_BLOCKS = 1024;

// 8 consecutive 16-bit elements <-> fp32
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  unpack2<BF16>(u.x, x[0], x[1]);
  unpack2<BF16>(u.y, x[2], x[3]);
  unpack2<BF16>(u.z, x[4], x[5]);
  unpack2<BF16>(u.w, x[6], x[7]);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                    pack2<BF16>(x[6], x[7]));
}

// A lane's part of one token's rotation: its 8 elements become x*cs + partner*sn. Split halves:
// the partner elements sit rot/16 lanes away (rot is a multiple of 16, so a lane lies wholly in
// the first half, the second, or behind both); pairs (2i, 2i+1) sit in the lane itself.
template <int D, bool INTER>
struct Turn {
  float cs[INTER ? 4 : 8], sn[INTER ? 4 : 8];
  int partner;

  // sign = 1 for the rotation, -1 for its transpose
  __device__ __forceinline__ void load(const RopeDev& rp, int pos, int l, int lane, float sign) {
    const int half = rp.rot >> 1, e = 8 * l;
    partner = lane;
#pragma unroll
    for (int i = 0; i < (INTER ? 4 : 8); ++i) cs[i] = 1.f, sn[i] = 0.f;
    if (e >= rp.rot) return;
    const float* row = rp.table + (size_t)pos * rp.rot;
    if constexpr (INTER) {
      const float4 c = *reinterpret_cast<const float4*>(row + e / 2);
      const float4 s = *reinterpret_cast<const float4*>(row + half + e / 2);
      cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
      sn[0] = sign * s.x, sn[1] = sign * s.y, sn[2] = sign * s.z, sn[3] = sign * s.w;
    } else {
      const bool second = e >= half;
      const float* c = row + (second ? e - half : e);
      const float4 c0 = *reinterpret_cast<const float4*>(c), c1 = *reinterpret_cast<const float4*>(c + 4);
      const float4 s0 = *reinterpret_cast<const float4*>(c + half), s1 = *reinterpret_cast<const float4*>(c + half + 4);
      const float sg = second ? sign : -sign;
      cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
      cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
      sn[0] = sg * s0.x, sn[1] = sg * s0.y, sn[2] = sg * s0.z, sn[3] = sg * s0.w;
      sn[4] = sg * s1.x, sn[5] = sg * s1.y, sn[6] = sg * s1.z, sn[7] = sg * s1.w;
      partner = second ? lane - half / 8 : lane + half / 8;
    }
  }
  // every lane of the warp calls this
  __device__ __forceinline__ void apply(float (&x)[8]) const {
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * cs[i] - b * sn[i];
        x[2 * i + 1] = b * cs[i] + a * sn[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * cs[i] + __shfl_sync(0xffffffffu, x[i], partner) * sn[i];
    }
  }
};

// sum over the lanes of a row (LPR consecutive lanes), the same in each of them
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct NormRopeParams {
  HeadsDev q, k, q_out, k_out;  // backward: inputs and their gradients (outputs)
  HeadsDev gq, gk;              // backward: gradients of the outputs
  const uint16_t *wq, *wk;
  float eps;
  RopeDev rope;
  const int* positions;
  int N;
  long long tokens;       // B * N
  int chunk, n_chunks;    // heads of q then k, `chunk` of them per warp
  float* part;            // backward: [block][2][D] sums of the weights' gradients
  int* status;
};

// y = R(p) (x r w): one warp per (token, chunk of heads).
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(ROW_THREADS) fa_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const long long unit = (long long)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5);
  const long long t = unit / p.n_chunks;
  if (t >= p.tokens) return;
  const int c = (int)(unit % p.n_chunks);
  const int b = (int)(t / p.N), n = (int)(t % p.N);
  const int pos = p.positions ? p.positions[t] : n;
  if (p.rope.rot && (pos < 0 || pos >= p.rope.length)) {
    if (lane == 0) atomicCAS(p.status, 0, FA_ERR_RANGE);
    return;
  }
  Turn<D, INTER> turn;
  turn.load(p.rope, pos, l, lane, 1.f);
  const int H = p.q.H + p.k.H, h_end = min((c + 1) * p.chunk, H);
  const uint16_t* qi = p.q.ptr + b * p.q.bs + n * p.q.ts + 8 * l;
  const uint16_t* ki = p.k.ptr + b * p.k.bs + n * p.k.ts + 8 * l;
  uint16_t* qo = p.q_out.ptr + b * p.q_out.bs + n * p.q_out.ts + 8 * l;
  uint16_t* ko = p.k_out.ptr + b * p.k_out.bs + n * p.k_out.ts + 8 * l;
  for (int h0 = c * p.chunk; h0 < h_end; h0 += GPW * ROW_UNROLL) {
    uint4 u[ROW_UNROLL];
#pragma unroll
    for (int i = 0; i < ROW_UNROLL; ++i) {
      const int h = h0 + i * GPW + sub;
      u[i] = make_uint4(0, 0, 0, 0);
      if (h < h_end)
        u[i] = *reinterpret_cast<const uint4*>(h < p.q.H ? qi + h * p.q.hs : ki + (h - p.q.H) * p.k.hs);
    }
#pragma unroll
    for (int i = 0; i < ROW_UNROLL; ++i) {
      const int h = h0 + i * GPW + sub;
      float x[8], w[8];
      unpack8<BF16>(u[i], x);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
      const uint16_t* wp = h < p.q.H ? p.wq : p.wk;
      uint4 wu = make_uint4(0, 0, 0, 0);
      if (h < h_end) wu = *reinterpret_cast<const uint4*>(wp + 8 * l);
      unpack8<BF16>(wu, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= r * w[e];
      turn.apply(x);
      if (h < h_end)
        *reinterpret_cast<uint4*>(h < p.q.H ? qo + h * p.q_out.hs : ko + (h - p.q.H) * p.k_out.hs) = pack8<BF16>(x);
    }
  }
}

// dx = r (u - x r mean(u x r)), u = R^T dy * w; the block's sums of R^T dy * x * r go to `part`.
// A fixed number of blocks walks the (token, chunk) units, so each sum has a fixed order.
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(ROW_THREADS) fa_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  __shared__ float sums[ROW_WARPS][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sub = lane / LPR;
  const int H = p.q.H + p.k.H;
  float aq[8] = {}, ak[8] = {}, wq[8], wk[8];
  uint4 wu = make_uint4(0, 0, 0, 0);
  if (p.q.H) wu = *reinterpret_cast<const uint4*>(p.wq + 8 * l);
  unpack8<BF16>(wu, wq);
  wu = make_uint4(0, 0, 0, 0);
  if (p.k.H) wu = *reinterpret_cast<const uint4*>(p.wk + 8 * l);
  unpack8<BF16>(wu, wk);
  const long long units = p.tokens * p.n_chunks, step = (long long)gridDim.x * ROW_WARPS;
  for (long long unit = (long long)blockIdx.x * ROW_WARPS + warp; unit < units; unit += step) {
    const long long t = unit / p.n_chunks;
    const int c = (int)(unit % p.n_chunks);
    const int b = (int)(t / p.N), n = (int)(t % p.N);
    const int pos = p.positions ? p.positions[t] : n;
    if (p.rope.rot && (pos < 0 || pos >= p.rope.length)) {
      if (lane == 0) atomicCAS(p.status, 0, FA_ERR_RANGE);
      continue;
    }
    Turn<D, INTER> turn;
    turn.load(p.rope, pos, l, lane, -1.f);
    const int h_end = min((c + 1) * p.chunk, H);
    const long long oq = b * p.q.bs + n * p.q.ts + 8 * l, ok = b * p.k.bs + n * p.k.ts + 8 * l;
    const long long ogq = b * p.gq.bs + n * p.gq.ts + 8 * l, ogk = b * p.gk.bs + n * p.gk.ts + 8 * l;
    const long long ooq = b * p.q_out.bs + n * p.q_out.ts + 8 * l, ook = b * p.k_out.bs + n * p.k_out.ts + 8 * l;
    for (int h0 = c * p.chunk; h0 < h_end; h0 += GPW * 2) {
      uint4 ux[2], ug[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = h0 + i * GPW + sub;
        ux[i] = ug[i] = make_uint4(0, 0, 0, 0);
        if (h < h_end) {
          const bool isq = h < p.q.H;
          const long long hk = h - p.q.H;
          ux[i] = *reinterpret_cast<const uint4*>(isq ? p.q.ptr + oq + h * p.q.hs : p.k.ptr + ok + hk * p.k.hs);
          ug[i] = *reinterpret_cast<const uint4*>(isq ? p.gq.ptr + ogq + h * p.gq.hs : p.gk.ptr + ogk + hk * p.gk.hs);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = h0 + i * GPW + sub;
        const bool isq = h < p.q.H;
        float x[8], g[8];
        unpack8<BF16>(ux[i], x);
        unpack8<BF16>(ug[i], g);
        turn.apply(g);
        float ss = 0.f, gx = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(x[e], x[e], ss);
          gx = fmaf(g[e] * (isq ? wq[e] : wk[e]), x[e], gx);
        }
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
        const float m = row_sum<LPR>(gx) * r * (1.f / D);  // mean(u x r)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xr = x[e] * r, gw = g[e] * xr;  // rows past h_end hold zeros
          if (isq) aq[e] += gw; else ak[e] += gw;
          x[e] = r * (g[e] * (isq ? wq[e] : wk[e]) - xr * m);
        }
        if (h < h_end)
          *reinterpret_cast<uint4*>(isq ? p.q_out.ptr + ooq + h * p.q_out.hs
                                        : p.k_out.ptr + ook + (long long)(h - p.q.H) * p.k_out.hs) = pack8<BF16>(x);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      aq[e] += __shfl_xor_sync(0xffffffffu, aq[e], o);
      ak[e] += __shfl_xor_sync(0xffffffffu, ak[e], o);
    }
    if (sub == 0) sums[warp][0][8 * l + e] = aq[e], sums[warp][1][8 * l + e] = ak[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += ROW_THREADS) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < ROW_WARPS; ++w) s += sums[w][i / D][i % D];
    p.part[(size_t)blockIdx.x * 2 * D + i] = s;
  }
}

// dw[set][c] = sum over blocks of part[block][set][c]: 32 columns x 32 slices of the blocks.
template <int D>
__global__ void __launch_bounds__(1024) fa_norm_rope_dw_kernel(const float* part, int blocks, float* dwq, float* dwk) {
  __shared__ float s[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float a = 0.f;
  for (int i = threadIdx.y; i < blocks; i += 32) a += part[(size_t)i * 2 * D + col];
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y) return;
  a = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) a += s[i][threadIdx.x];
  float* dst = col < D ? dwq : dwk;
  if (dst) dst[col % D] = a;
}

// ------------------------------------------------------------------------------ append
struct AppendParams {
  HeadsDev k, v;
  uint16_t *kp, *vp;  // pages
  long long page_stride, head_stride, token_stride;
  int num_pages, page_size;
  const int *cu, *lens, *table;
  int table_stride, B, T;
  RopeDev rope;
  int chunk, n_chunks;  // heads of k then v, `chunk` of them per warp
  int* status;
};

// The sequence whose new tokens hold row t (cu[b] <= t < cu[b+1]), or -1; the warp's 32 lanes
// look at 32 places at a time. cu has B + 1 entries that do not decrease.
__device__ __forceinline__ int find_sequence(const int* cu, int B, int t, int lane) {
  int lo = 0, n = B + 1;  // the answer + 1 = number of entries <= t, all of them in [0, lo + n)
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;  // last entry of this lane's part
    const bool le = i < lo + n && cu[i] <= t;
    const int parts = __popc(__ballot_sync(0xffffffffu, le));
    const int skip = parts * step;
    lo += skip;
    n = min(step - 1, n - skip);
  }
  return lo >= 1 && lo <= B ? lo - 1 : -1;
}

// One warp per (token, chunk of heads): the token's sequence, position, page and slot, then its
// rows of k (rotated) and v (copied).
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(ROW_THREADS) fa_paged_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const long long unit = (long long)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5);
  const int t = (int)(unit / p.n_chunks);
  if (t >= p.T) return;
  const int c = (int)(unit % p.n_chunks);
  const int b = find_sequence(p.cu, p.B, t, lane);
  if (b < 0) return;
  const int pos = p.lens[b] - (p.cu[b + 1] - t);
  int page = -1;
  const bool in = pos >= 0 && pos / p.page_size < p.table_stride && (!p.rope.rot || pos < p.rope.length);
  if (in) page = p.table[(size_t)b * p.table_stride + pos / p.page_size];
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0) atomicCAS(p.status, 0, FA_ERR_RANGE);
    return;
  }
  const long long base = page * p.page_stride + (long long)(pos % p.page_size) * p.token_stride + 8 * l;
  Turn<D, INTER> turn;
  turn.load(p.rope, pos, l, lane, 1.f);
  const int Hk = p.k.H, h_end = min((c + 1) * p.chunk, 2 * Hk);
  const uint16_t* ki = p.k.ptr + t * p.k.ts + 8 * l;
  const uint16_t* vi = p.v.ptr + t * p.v.ts + 8 * l;
  for (int h0 = c * p.chunk; h0 < h_end; h0 += GPW * ROW_UNROLL) {
    uint4 u[ROW_UNROLL];
#pragma unroll
    for (int i = 0; i < ROW_UNROLL; ++i) {
      const int h = h0 + i * GPW + sub;
      u[i] = make_uint4(0, 0, 0, 0);
      if (h < h_end) u[i] = *reinterpret_cast<const uint4*>(h < Hk ? ki + h * p.k.hs : vi + (h - Hk) * p.v.hs);
    }
#pragma unroll
    for (int i = 0; i < ROW_UNROLL; ++i) {
      const int h = h0 + i * GPW + sub;
      if (p.rope.rot && h0 + i * GPW < Hk) {  // a warp's rows of this step may straddle k and v
        float x[8];
        unpack8<BF16>(u[i], x);
        turn.apply(x);
        if (h < Hk) u[i] = pack8<BF16>(x);
      }
      if (h < h_end)
        *reinterpret_cast<uint4*>((h < Hk ? p.kp + h * p.head_stride : p.vp + (h - Hk) * p.head_stride) + base) = u[i];
    }
  }
}

}  // namespace fa
