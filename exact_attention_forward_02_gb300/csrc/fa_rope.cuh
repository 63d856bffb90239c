// fa_rope.cuh -- per-row kernels over query, key and value heads: RMS norm + position rotation
// (forward and backward) and the append to a paged cache. Included by fa_decoder.cu.
//
// All of them read and write each row of d 16-bit elements once and are bound by HBM. A row is
// held by d/8 lanes, 8 elements each: 2 (d = 128) or 4 (d = 64) groups of lanes to a warp. A group
// works on ONE token and walks its heads, so that its lanes load their angles of the rotation
// table, and work out their addresses, once for all of them. (A warp per token, its groups side by
// side on the token's heads, paid for that 2 or 4 times as often: 10.2 us for 16384 tokens of 2 + 1
// heads, d = 64.) A lane holds both elements of each of its 4 pairs (A and B below), so the rotation
// needs no exchange between lanes, and works on them two at a time (f32x2).
//
// Every kernel here is launched so that its blocks may be set up while the previous kernel of the
// stream still runs (launch_dependent in fa_decoder.cu): it waits for that kernel's results
// (wait_previous_grid) before it reads or writes global memory.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "fa_decoder.h"
#include "sm103_ptx.cuh"

namespace fa {

// Debug builds (FA_DEBUG) check the places of tile copies, partial states, rows and weights; one outside records
// FA_ERR_BOUNDS in the status word of the kernel's parameters. Stores, and the join of an item whose pieces it
// concerns, are then skipped; a tile copy is only recorded (TMA reads zeros outside, and its barrier expects
// the bytes). Release builds compile it out.
template <typename P>
__device__ __forceinline__ bool in_bounds(const P& p, bool ok) {
#ifdef FA_DEBUG
  if (!ok) atomicCAS(p.status, 0, FA_ERR_BOUNDS);
  return ok;
#else
  (void)p, (void)ok;
  return true;
#endif
}

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
constexpr int ROW_MIN_WARPS = 16;      // warps per SM below which heads are shared out further
constexpr int ROW_BWD_MAX_BLOCKS = 1024;

// 8 consecutive 16-bit elements from fp32
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                    pack2<BF16>(x[6], x[7]));
}

// A lane's 8 elements of a row as 4 pairs (A_i, B_i) in fp32, two pairs to a register pair.
struct Pairs {
  uint64_t a[2], b[2];
};
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// Where a lane's pairs stand in a row, and a token's rotation of them. Pairs (2i, 2i+1): the lane
// holds 8 consecutive elements. Split halves (i, i + rot/2): lane l < rot/8 holds elements
// 4l .. 4l+3 (A) and rot/2 + 4l .. (B); the other lanes hold 8 consecutive elements behind rot,
// which pass through as they are, whatever stands beside them. rot is a multiple of 16; FULL: it is
// D, and no lane has to choose between its turned and its own elements (a choice in every row costs
// the gradients 2 us of 88).
template <int D, bool BF16, bool INTER, bool FULL>
struct Lane {
  int l, ea, eb;  // lane of the row, first elements of its two runs of 4
  bool turns;     // its pairs are rotated
  uint64_t c[2], s[2];

  __device__ __forceinline__ void place(int lane, int rot) {
    l = lane % (D / 8);
    turns = FULL || 8 * l < rot;
    const bool split = !INTER && turns;
    ea = split ? 4 * l : 8 * l;
    eb = split ? 4 * l + rot / 2 : 8 * l + 4;
  }
  // index in the row of A_i and B_i
  __device__ __forceinline__ int at(int i, bool second) const {
    return INTER ? 8 * l + 2 * i + second : (second ? eb : ea) + i;
  }
  // sign = 1 for the rotation, -1 for its transpose
  __device__ __forceinline__ void angles(const RopeDev& rp, int pos, float sign, bool known) {
    c[0] = c[1] = f2(1.f, 1.f);
    s[0] = s[1] = 0;
    if (!turns || !known) return;
    const float* row = rp.table + (size_t)pos * rp.rot + 4 * l;
    const float4 x = *reinterpret_cast<const float4*>(row), y = *reinterpret_cast<const float4*>(row + rp.rot / 2);
    c[0] = f2(x.x, x.y), c[1] = f2(x.z, x.w);
    s[0] = f2(sign * y.x, sign * y.y), s[1] = f2(sign * y.z, sign * y.w);
  }
  __device__ __forceinline__ uint4 load(const uint16_t* row) const {
    if constexpr (INTER) return *reinterpret_cast<const uint4*>(row + 8 * l);
    const uint2 x = *reinterpret_cast<const uint2*>(row + ea), y = *reinterpret_cast<const uint2*>(row + eb);
    return make_uint4(x.x, x.y, y.x, y.y);
  }
  __device__ __forceinline__ void store(uint16_t* row, const uint4& u) const {
    if constexpr (INTER) {
      *reinterpret_cast<uint4*>(row + 8 * l) = u;
    } else {
      *reinterpret_cast<uint2*>(row + ea) = make_uint2(u.x, u.y);
      *reinterpret_cast<uint2*>(row + eb) = make_uint2(u.z, u.w);
    }
  }
  __device__ __forceinline__ Pairs unpack(const uint4& u) const {
    float x0, x1, x2, x3, y0, y1, y2, y3;
    unpack2<BF16>(u.x, x0, x1);
    unpack2<BF16>(u.y, x2, x3);
    unpack2<BF16>(u.z, y0, y1);
    unpack2<BF16>(u.w, y2, y3);
    if constexpr (INTER) return Pairs{{f2(x0, x2), f2(y0, y2)}, {f2(x1, x3), f2(y1, y3)}};
    return Pairs{{f2(x0, x1), f2(x2, x3)}, {f2(y0, y1), f2(y2, y3)}};
  }
  __device__ __forceinline__ uint4 pack(const Pairs& v) const {
    if constexpr (INTER)
      return make_uint4(pack2<BF16>(lo_of(v.a[0]), lo_of(v.b[0])), pack2<BF16>(hi_of(v.a[0]), hi_of(v.b[0])),
                        pack2<BF16>(lo_of(v.a[1]), lo_of(v.b[1])), pack2<BF16>(hi_of(v.a[1]), hi_of(v.b[1])));
    return make_uint4(pack2<BF16>(lo_of(v.a[0]), hi_of(v.a[0])), pack2<BF16>(lo_of(v.a[1]), hi_of(v.a[1])),
                      pack2<BF16>(lo_of(v.b[0]), hi_of(v.b[0])), pack2<BF16>(lo_of(v.b[1]), hi_of(v.b[1])));
  }
  // (A, B) -> (A cos - B sin, B cos + A sin)
  __device__ __forceinline__ void turn(Pairs& v) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t minus = s[i] ^ 0x8000000080000000ull;
      const uint64_t a = f2_fma(v.a[i], c[i], f2_mul(v.b[i], minus));
      const uint64_t b = f2_fma(v.b[i], c[i], f2_mul(v.a[i], s[i]));
      v.a[i] = turns ? a : v.a[i];
      v.b[i] = turns ? b : v.b[i];
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
  HeadsDev x[2], y[2];  // q and k: inputs, and outputs (backward: the inputs' gradients)
  HeadsDev g[2];        // backward: gradients of the outputs
  const uint16_t* w[2];
  float eps;
  RopeDev rope;
  const int* positions;
  int N, tokens;        // tokens = B * N
  uint32_t units;       // of a warp: ceil(tokens / groups of lanes) * n_chunks
  int chunk, n_chunks;  // heads of q then k, `chunk` of them per unit
  float* part;          // backward: [block][2][D] sums of the weights' gradients
  int* status;
};

__device__ __forceinline__ float sum4(const uint64_t (&v)[2]) {
  return (lo_of(v[0]) + hi_of(v[0])) + (lo_of(v[1]) + hi_of(v[1]));
}

// A warp's unit: heads [c, c + chunk) of q's, then k's, of one token for each group of lanes.
// 32-bit divisions: the host checks that the units fit.
template <int GPW>
struct RowUnit {
  int t, b, n, c, pos;
  bool alive;  // the group has a token, and its position a row of the table
  __device__ __forceinline__ RowUnit(const NormRopeParams& p, uint32_t unit, int sub) {
    const uint32_t tg = p.n_chunks == 1 ? unit : unit / (uint32_t)p.n_chunks;
    c = (int)(unit - tg * p.n_chunks) * p.chunk;
    t = (int)(tg * GPW) + sub;
    alive = t < p.tokens;
    if (!alive) t = p.tokens - 1;
    b = (uint32_t)t / (uint32_t)p.N;
    n = t - b * p.N;
  }
  __device__ __forceinline__ void locate(const NormRopeParams& p, int l) {
    pos = p.positions ? p.positions[t] : n;
    if (alive && p.rope.rot && (pos < 0 || pos >= p.rope.length)) {
      if (l == 0) atomicCAS(p.status, 0, FA_ERR_RANGE);
      alive = false;
    }
  }
  // A group without a token takes the rows of one that has one (`some`: the lanes of those), so that
  // what it works out and drops is no worse than that token's own: its own rows may hold anything.
  __device__ __forceinline__ void borrow(uint32_t some) {
    const int from = alive ? threadIdx.x & 31 : __ffs(some) - 1;
    t = __shfl_sync(0xffffffffu, t, from);
    b = __shfl_sync(0xffffffffu, b, from);
    n = __shfl_sync(0xffffffffu, n, from);
  }
  // the unit's heads of a set whose first head is `first`
  __device__ __forceinline__ int begin(int first) const { return max(c - first, 0); }
  __device__ __forceinline__ int end(const NormRopeParams& p, int first, int H) const { return min(c + p.chunk - first, H); }
  __device__ __forceinline__ uint16_t* row(const HeadsDev& x, int h) const {
    return x.ptr + b * x.bs + n * x.ts + h * x.hs;
  }
};

// y = R(p) (x r w): one warp per unit. 4 rows in flight per group and 64 registers, so that 32 warps
// fit an SM. 16384 tokens of 32 + 8 heads, d 128: 56 us, 6.1 TB/s of the copy's 6.8.
template <int D, bool BF16, bool INTER, bool FULL>
__global__ void __launch_bounds__(ROW_THREADS, 4) fa_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR;
  const uint32_t unit = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  RowUnit<GPW> at(p, unit, sub);
  Lane<D, BF16, INTER, FULL> ln;
  ln.place(lane, p.rope.rot);
  launch_dependents();
  wait_previous_grid();
  at.locate(p, ln.l);
  if (!__any_sync(0xffffffffu, at.alive)) return;
  ln.angles(p.rope, at.pos, 1.f, at.alive);
#pragma unroll 1
  for (int set = 0; set < 2; ++set) {
    const HeadsDev &in = p.x[set], &out = p.y[set];
    const int first = set ? p.x[0].H : 0, h_begin = at.begin(first), h_end = at.end(p, first, in.H);
    if (h_begin >= h_end) continue;
    const Pairs w = ln.unpack(ln.load(p.w[set]));
    const uint16_t* src = at.row(in, h_begin);
    uint16_t* dst = at.row(out, h_begin);
    auto finish = [&](const uint4& u, uint16_t* to) {
      Pairs x = ln.unpack(u);
      uint64_t sq[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) sq[e] = f2_fma(x.b[e], x.b[e], f2_mul(x.a[e], x.a[e]));
      const float r = rsqrtf(row_sum<LPR>(sum4(sq)) * (1.f / D) + p.eps);
      const uint64_t r2 = f2(r, r);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x.a[e] = f2_mul(x.a[e], f2_mul(w.a[e], r2));
        x.b[e] = f2_mul(x.b[e], f2_mul(w.b[e], r2));
      }
      ln.turn(x);
      if (at.alive) ln.store(to, ln.pack(x));
    };
    int left = h_end - h_begin;  // heads
#pragma unroll 1
    for (; left >= ROW_UNROLL; left -= ROW_UNROLL) {
      uint4 u[ROW_UNROLL];
#pragma unroll
      for (int i = 0; i < ROW_UNROLL; ++i, src += in.hs) u[i] = ln.load(src);
#pragma unroll
      for (int i = 0; i < ROW_UNROLL; ++i, dst += out.hs) finish(u[i], dst);
    }
#pragma unroll 1
    for (; left > 0; --left, src += in.hs, dst += out.hs) finish(ln.load(src), dst);
  }
}

// dx = r (u - x r mean(u x r)), u = R^T dy * w; the block's sums of R^T dy * x * r go to `part`.
// A group without a token adds g = 0 times a borrowed row to them (zeroing its x and r in the loop as
// well costs 1 us of 88). A fixed number of blocks walks the units, so each sum has a fixed order. Four rows of both
// tensors in flight per lane group and two blocks per SM (128 registers; 1, 3 and 4 blocks: 127,
// 108 and 123 us against 87). 16384 tokens of 32 + 8 heads, d 128: 88 us with the sums, 5.8 TB/s.
template <int D, bool BF16, bool INTER, bool FULL>
__global__ void __launch_bounds__(ROW_THREADS, 2) fa_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  __shared__ float sums[ROW_WARPS][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR;
  Lane<D, BF16, INTER, FULL> ln;
  ln.place(lane, p.rope.rot);
  launch_dependents();
  wait_previous_grid();
  Pairs dw[2] = {};
#pragma unroll 1
  for (uint32_t unit = blockIdx.x * ROW_WARPS + warp; unit < p.units; unit += gridDim.x * ROW_WARPS) {
    RowUnit<GPW> at(p, unit, sub);
    at.locate(p, ln.l);
    const uint32_t some = __ballot_sync(0xffffffffu, at.alive);
    if (!some) continue;
    at.borrow(some);
    ln.angles(p.rope, at.pos, -1.f, at.alive);
#pragma unroll
    for (int set = 0; set < 2; ++set) {
      const HeadsDev &in = p.x[set], &gr = p.g[set], &out = p.y[set];
      const int first = set ? p.x[0].H : 0, h_begin = at.begin(first), h_end = at.end(p, first, in.H);
      if (h_begin >= h_end) continue;
      const Pairs w = ln.unpack(ln.load(p.w[set]));
      const uint16_t* src = at.row(in, h_begin);
      const uint16_t* gsrc = at.row(gr, h_begin);
      uint16_t* dst = at.row(out, h_begin);
      auto load_g = [&]() { return at.alive ? ln.load(gsrc) : make_uint4(0, 0, 0, 0); };  // adds nothing to dw
      auto finish = [&](const uint4& ux, const uint4& ug, uint16_t* to) {
        Pairs x = ln.unpack(ux), g = ln.unpack(ug), u;
        ln.turn(g);
        uint64_t sq[2], gx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sq[e] = f2_fma(x.b[e], x.b[e], f2_mul(x.a[e], x.a[e]));
          u.a[e] = f2_mul(g.a[e], w.a[e]);
          u.b[e] = f2_mul(g.b[e], w.b[e]);
          gx[e] = f2_fma(u.b[e], x.b[e], f2_mul(u.a[e], x.a[e]));
        }
        const float r = rsqrtf(row_sum<LPR>(sum4(sq)) * (1.f / D) + p.eps);
        const float m = row_sum<LPR>(sum4(gx)) * r * (-1.f / D);  // - mean(u x r)
        const uint64_t r2 = f2(r, r), m2 = f2(m, m);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint64_t xa = f2_mul(x.a[e], r2), xb = f2_mul(x.b[e], r2);
          dw[set].a[e] = f2_fma(g.a[e], xa, dw[set].a[e]);
          dw[set].b[e] = f2_fma(g.b[e], xb, dw[set].b[e]);
          x.a[e] = f2_mul(f2_fma(xa, m2, u.a[e]), r2);
          x.b[e] = f2_mul(f2_fma(xb, m2, u.b[e]), r2);
        }
        if (at.alive) ln.store(to, ln.pack(x));
      };
      int left = h_end - h_begin;  // heads
#pragma unroll 1
      for (; left >= ROW_UNROLL; left -= ROW_UNROLL) {
        uint4 ux[ROW_UNROLL], ug[ROW_UNROLL];
#pragma unroll
        for (int i = 0; i < ROW_UNROLL; ++i, src += in.hs, gsrc += gr.hs) {
          ux[i] = ln.load(src);
          ug[i] = load_g();
        }
#pragma unroll
        for (int i = 0; i < ROW_UNROLL; ++i, dst += out.hs) finish(ux[i], ug[i], dst);
      }
#pragma unroll 1
      for (; left > 0; --left, src += in.hs, gsrc += gr.hs, dst += out.hs) finish(ln.load(src), load_g(), dst);
    }
  }
#pragma unroll
  for (int set = 0; set < 2; ++set)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t v = i < 4 ? dw[set].a[i >> 1] : dw[set].b[(i >> 1) - 2];
      float x = i & 1 ? hi_of(v) : lo_of(v);
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (sub == 0) sums[warp][set][ln.at(i & 3, i >= 4)] = x;
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
  launch_dependents();
  wait_previous_grid();
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
  uint32_t units;       // of a warp: ceil(T / groups of lanes) * n_chunks
  int chunk, n_chunks;  // heads of k then v, `chunk` of them per unit
  int* status;
};

// A sequence's rows lie within the T that there are (the attention passes over the others as well).
__device__ __forceinline__ bool rows_fit(const AppendParams& p, int begin, int end) {
  return begin >= 0 && end >= begin && end <= p.T;
}

// The sequence whose new tokens hold row t (cu[b] <= t < cu[b+1]), or -1; the warp's 32 lanes
// look at 32 places at a time. cu has B + 1 entries that do not decrease (if they do: any sequence, or -1).
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

// Bound by HBM: 65536 tokens of 8 heads, d 128, in 84 us (the copy's rate), 29582 ragged ones in 41;
// 64 single tokens in 2.9 us. One warp per unit: each group's token's sequence, position, page and slot, then its rows of k
// (rotated) and v (copied).
template <int D, bool BF16, bool INTER, bool FULL>
__global__ void __launch_bounds__(ROW_THREADS, 4) fa_paged_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR;
  const uint32_t unit = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5);
  if (blockIdx.x == gridDim.x - 1) {  // looks over the offsets; the others skip what does not fit them
    launch_dependents();
    wait_previous_grid();
    bool bad = false;
#pragma unroll 4
    for (int i = threadIdx.x; i < p.B; i += ROW_THREADS) bad |= !rows_fit(p, p.cu[i], p.cu[i + 1]);
    if (bad) atomicCAS(p.status, 0, FA_ERR_RANGE);
    return;
  }
  if (unit >= p.units) return;
  const uint32_t tg = unit / (uint32_t)p.n_chunks;
  const int c = (int)(unit - tg * p.n_chunks), t0 = (int)(tg * GPW), t = t0 + sub;
  Lane<D, BF16, INTER, FULL> ln;
  ln.place(lane, p.rope.rot);
  launch_dependents();
  wait_previous_grid();
  int b = -1;
#pragma unroll
  for (int i = 0; i < GPW; ++i) {
    const int bi = find_sequence(p.cu, p.B, min(t0 + i, p.T - 1), lane);
    if (i == sub && t < p.T) b = bi;
  }
  int pos = 0, page = -1;
  if (b >= 0) {
    const int begin = p.cu[b], end = p.cu[b + 1];
    pos = p.lens[b] - (end - t);
    if (!rows_fit(p, begin, end) || t < begin || t >= end) b = -1;
  }
  if (b >= 0) {
    const bool in = pos >= 0 && pos / p.page_size < p.table_stride && (!p.rope.rot || pos < p.rope.length);
    if (in) page = p.table[(size_t)b * p.table_stride + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      if (ln.l == 0) atomicCAS(p.status, 0, FA_ERR_RANGE);
      b = -1;
    }
  }
  if (b < 0) return;  // nothing below is shared between lanes
  const long long base = page * p.page_stride + (long long)(pos % p.page_size) * p.token_stride;
  ln.angles(p.rope, pos, 1.f, true);
#pragma unroll 1
  for (int set = 0; set < 2; ++set) {
    const HeadsDev& in = set ? p.v : p.k;
    const int first = set ? p.k.H : 0;
    const int h_begin = max(c * p.chunk - first, 0), h_end = min((c + 1) * p.chunk - first, in.H);
    if (h_begin >= h_end) continue;
    const uint16_t* src = in.ptr + t * in.ts + h_begin * in.hs;
    uint16_t* dst = (set ? p.vp : p.kp) + base + h_begin * p.head_stride;
    const bool turned = set == 0 && p.rope.rot;
    auto finish = [&](uint4 u, uint16_t* to) {
      if (turned) {
        Pairs x = ln.unpack(u);
        ln.turn(x);
        const uint4 w = ln.pack(x);
        u = ln.turns ? w : u;  // bit by bit where it passes through
      }
      ln.store(to, u);
    };
    int left = h_end - h_begin;  // heads
#pragma unroll 1
    for (; left >= ROW_UNROLL; left -= ROW_UNROLL) {
      uint4 u[ROW_UNROLL];
#pragma unroll
      for (int i = 0; i < ROW_UNROLL; ++i, src += in.hs) u[i] = ln.load(src);
#pragma unroll
      for (int i = 0; i < ROW_UNROLL; ++i, dst += p.head_stride) finish(u[i], dst);
    }
#pragma unroll 1
    for (; left > 0; --left, src += in.hs, dst += p.head_stride) finish(ln.load(src), dst);
  }
}

}  // namespace fa
