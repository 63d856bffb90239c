// fa_append8.cuh -- new keys (rotated) and values into a paged cache held in 8 bits.
// Included by fa_append8.cu.
//
// A page of a key head is held as x = s c, c in E4M3 and s one scale of fp32. For the new tokens of a
// page, a = max |x| over their (rotated) rows asks for s_new = the smallest power of two >= a / 448;
// with older tokens in the page its scale becomes s = max(s_old, s_new), else s_new. A power of two
// costs E4M3 no precision (its 4 bits are relative to the value), and codes held under a smaller scale
// are then rounded anew exactly, but for what falls among the subnormal numbers (below 2^-14 of the
// largest): so a page's codes hardly depend on how its tokens were cut into calls.
//
// Work: a unit is (sequence, page it gets tokens into, head of k or of v), one to W warps, which hold
// the unit's rows in registers between the maximum and the rounding. No atomics: a page belongs to one
// unit. Places for pages, and whose they are: append8_places.h.
//
// HBM would allow a time of 3 d bytes an element row; what bounds it is the issue of instructions (69 % of the slots,
// about 200 instructions to 256 elements, a warp's part of the search among them) and the one chain of a unit's loads,
// search to scale. 29582 ragged tokens of 8 heads, d 128, pages of 64, fp16: 57 us, 3.4 TB/s of 6.8. Units that walk
// several heads of a page, one search for many rows, took 74 to 82. 64 single tokens: 3.5 us, latency.
#pragma once

#include "append8_places.h"
#include "fa_rope.cuh"

namespace fa {

struct Append8Params {
  HeadsDev k, v;
  uint8_t *kp, *vp;
  float *ks, *vs;  // [num_pages][Hkv]
  long long page_stride, head_stride, token_stride;
  int num_pages, page_size, Hkv;
  const int *cu, *lens, *table;
  int table_stride, B, T;
  long long units;  // places for pages, times the heads of k and of v
  RopeDev rope;
  int* status;
};

constexpr uint32_t APPEND8_LEAST = 27u << 23;      // 2^-100, of a page of zeros

// as the 16-bit append has it
__device__ __forceinline__ bool rows_fit(int begin, int end, int T) { return begin >= 0 && end >= begin && end <= T; }
// (the warp's 32 lanes look at 32 sequences at a time)
__device__ __forceinline__ int sequence_of_place(const Append8Params& p, uint32_t place, int lane) {
  return search_places(p.B, [&](int lo, int step, int end) {
    const int i = lo + (lane + 1) * step - 1;
    const bool le = i < end && first_place(p.cu[i], p.page_size, i) <= place;
    return __popc(__ballot_sync(0xffffffffu, le));
  });
}

// ROWS: rows that a lane holds between the two passes
template <int D, bool BF16, bool INTER, bool FULL, int W, int ROWS>
__global__ void __launch_bounds__(ROW_THREADS, ROWS > 4 ? 2 : 4) fa_paged_append8_kernel(const __grid_constant__ Append8Params p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR, TURN = W * GPW;  // lanes of a row, rows of a warp, of a unit's turn
  __shared__ float tops[2][ROW_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR, wu = warp % W;
  if (blockIdx.x == gridDim.x - 1) {  // looks over the offsets; the others skip what does not fit them
    launch_dependents();
    wait_previous_grid();
    bool bad = false;
#pragma unroll 4
    for (int i = threadIdx.x; i < p.B; i += ROW_THREADS) bad |= !rows_fit(p.cu[i], p.cu[i + 1], p.T);
    if (bad) atomicCAS(p.status, 0, FA_ERR_RANGE);
    return;
  }
  const long long unit = (long long)blockIdx.x * (ROW_WARPS / W) + warp / W;
  bool alive = unit < p.units;
  const int heads = 2 * p.Hkv;
  const uint32_t place = alive ? (uint32_t)(unit / heads) : 0u;
  const int hs = alive ? (int)(unit - (long long)place * heads) : 0;
  const bool is_v = hs >= p.Hkv;
  const int h = is_v ? hs - p.Hkv : hs;
  const HeadsDev& in = is_v ? p.v : p.k;
  const bool turned = !is_v && p.rope.rot;
  Lane<D, BF16, INTER, FULL> ln;
  ln.place(lane, p.rope.rot);
  launch_dependents();
  wait_previous_grid();
  const int b = sequence_of_place(p, place, lane);
  int begin = 0, p0 = 0, s0 = 0, s1 = 0, at = 0, page = -1;
  alive = alive && b >= 0;
  if (alive) {
    begin = p.cu[b];
    const int end = p.cu[b + 1], len = p.lens[b];
    const Piece x = piece_of(place, b, begin, end, len, p.T, p.page_size);
    if (x.early && lane == 0) atomicCAS(p.status, 0, FA_ERR_RANGE);  // tokens before position 0
    alive = x.alive;
    if (alive) {
      p0 = len - (end - begin), at = x.at, s0 = x.s0, s1 = x.s1;
      const long long from = (long long)at * p.page_size;
      // tokens behind the rotation table are skipped
      const int told = p.rope.rot ? (int)min((long long)s1, max(p.rope.length - from, 0ll)) : s1;
      bool bad = told < s1;
      s1 = told;
      if (at < p.table_stride) page = p.table[(size_t)b * p.table_stride + at];
      if (page < 0 || page >= p.num_pages) bad = true, alive = false;
      if (bad && lane == 0) atomicCAS(p.status, 0, FA_ERR_RANGE);
      alive = alive && s0 < s1;
      // the slots that are written, and the rows that go there
      alive = alive && in_bounds(p, s0 >= 0 && s1 <= p.page_size && h < p.Hkv && from + s0 >= p0 && from + s1 - p0 <= end - begin);
    }
  }
  const int pos0 = alive ? at * p.page_size : 0;  // of the page's first slot
  const uint16_t* src = in.ptr + (long long)h * in.hs + ((long long)begin + pos0 - p0) * in.ts;  // of that slot
  uint8_t* dst = (is_v ? p.vp : p.kp) + (long long)page * p.page_stride + (long long)h * p.head_stride;
  float* scale_at = (is_v ? p.vs : p.ks) + (long long)page * p.Hkv + h;
  const float s_old = alive && s0 > 0 ? *scale_at : 0.f;

  // a row's elements, rotated, and the maximum of their sizes (of those that are finite)
  auto load = [&](int slot) { return ln.load(src + (long long)slot * in.ts); };
  auto values = [&](const uint4& u, int slot) {
    Pairs x = ln.unpack(u);
    if (turned) {
      ln.angles(p.rope, pos0 + slot, 1.f, true);
      ln.turn(x);
    }
    return x;
  };
  float top = 0.f;
  bool wild = false;  // there are infinities: they become NaN first (a maximum passes over NaN)
  auto tame = [&](Pairs& x) {
    auto one = [&](uint64_t v) {
      const float a = lo_of(v), b = hi_of(v);
      return f2(a + (a - a), b + (b - b));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) x.a[i] = one(x.a[i]), x.b[i] = one(x.b[i]);
  };
  auto far = [&](int slot) {
    Pairs x = values(load(slot), slot);
    if (wild) tame(x);
    return x;
  };
  auto grow = [&](const Pairs& x) {
    auto one = [&](float v) { top = fmaxf(top, fabsf(v)); };
#pragma unroll
    for (int i = 0; i < 2; ++i) one(lo_of(x.a[i])), one(hi_of(x.a[i])), one(lo_of(x.b[i])), one(hi_of(x.b[i]));
  };
  auto put = [&](int slot, const Pairs& x, float inv) {
    auto q = [&](float v) { return v * inv; };
    uint8_t* row = dst + (long long)slot * p.token_stride;
    if constexpr (INTER) {
      const uint32_t w0 = pack4_e4m3(q(lo_of(x.a[0])), q(lo_of(x.b[0])), q(hi_of(x.a[0])), q(hi_of(x.b[0])));
      const uint32_t w1 = pack4_e4m3(q(lo_of(x.a[1])), q(lo_of(x.b[1])), q(hi_of(x.a[1])), q(hi_of(x.b[1])));
      *reinterpret_cast<uint2*>(row + 8 * ln.l) = make_uint2(w0, w1);
    } else {
      *reinterpret_cast<uint32_t*>(row + ln.ea) =
          pack4_e4m3(q(lo_of(x.a[0])), q(hi_of(x.a[0])), q(lo_of(x.a[1])), q(hi_of(x.a[1])));
      *reinterpret_cast<uint32_t*>(row + ln.eb) =
          pack4_e4m3(q(lo_of(x.b[0])), q(hi_of(x.b[0])), q(lo_of(x.b[1])), q(hi_of(x.b[1])));
    }
  };

  const int row0 = s0 + wu * GPW + sub, rows_held = ROWS * TURN;
  Pairs held[ROWS];
  if (alive) {
    uint4 u[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
      if (row0 + j * TURN < s1) u[j] = load(row0 + j * TURN);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      if (row0 + j * TURN >= s1) continue;
      held[j] = values(u[j], row0 + j * TURN);
      grow(held[j]);
    }
#pragma unroll 2
    for (int s = row0 + rows_held; s < s1; s += TURN) grow(far(s));  // (pages too large to be held)
  }
  auto join = [&](int set) {  // over the unit's warps
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if constexpr (W > 1) {
      if (lane == 0) tops[set][warp] = top;
      named_bar_sync(1 + warp / W, W * 32);
#pragma unroll
      for (int i = 0; i < W; ++i) top = fmaxf(top, tops[set][warp / W * W + i]);
    }
  };
  join(0);
  if (!alive) return;
  if (top > 3.402823466e38f) {
    wild = true;
    top = 0.f;
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
      if (row0 + j * TURN < s1) tame(held[j]), grow(held[j]);
#pragma unroll 1
    for (int s = row0 + rows_held; s < s1; s += TURN) grow(far(s));
    join(1);
  }
  // the smallest power of two that is not below top / 448: 448 = 1.75 2^8
  const uint32_t bits = (__float_as_uint(top) + 0x1fffffu) >> 23 << 23;
  float s = __uint_as_float(bits > APPEND8_LEAST + (8u << 23) ? bits - (8u << 23) : APPEND8_LEAST);
  if (s0 > 0 && s_old >= s) s = s_old;
  const float inv = 1.f / s;
#pragma unroll
  for (int j = 0; j < ROWS; ++j)
    if (row0 + j * TURN < s1) put(row0 + j * TURN, held[j], inv);
#pragma unroll 2
  for (int x = row0 + rows_held; x < s1; x += TURN) put(x, far(x), inv);
  if (s0 > 0 && s > s_old) {  // the older tokens' codes under the larger scale
    const float ratio = s_old * inv;
    for (int x = wu * GPW + sub; x < s0; x += TURN) {
      uint2* row = reinterpret_cast<uint2*>(dst + (long long)x * p.token_stride + 8 * ln.l);
      uint2 c = *row;
      auto again = [&](uint32_t v) {
        uint32_t a, e;
        float f[4];
        unpack4_e4m3(v, a, e);
        unpack2<false>(a, f[0], f[1]);
        unpack2<false>(e, f[2], f[3]);
        return pack4_e4m3(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
      };
      *row = make_uint2(again(c.x), again(c.y));
    }
  }
  if (lane == 0 && wu == 0 && (s0 == 0 || s > s_old)) *scale_at = s;
}

}  // namespace fa
