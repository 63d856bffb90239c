// fa_evict.cuh -- each key head's cached tokens cut to a budget: the most recent ones and those of the
// highest weight stay, moved together in order, in place. Included by fa_evict.cu.
//
// Kernel 1, a block for each (sequence, key head): the border weight is found by a radix select over the
// weights in the order of their bits (11, 11 and 10 bits, a histogram in shared memory each), ties go to
// the lowest positions, and the kept positions are listed in order: each warp counts its own run of
// positions, one scan over the warps, each warp writes its own. 8-bit caches: the scale of a page becomes the
// largest of those that its tokens come from, and each token's ratio is listed.
// Kernel 2 moves rows: token j of the kept ones comes from position src(j) >= j. A block takes some
// 16-byte columns of one head's rows of K or V (or its weights) and walks them in order: columns do not
// meet, and a round's stores go to places below every later round's sources, so that one barrier a round, between
// its loads and its stores, makes the move safe in place. Bound by HBM where there are heads enough.
#pragma once

#include "fa_rope.cuh"

namespace fa {
namespace evict {

constexpr int SELECT_THREADS = 1024, SELECT_WARPS = 32;
constexpr int BINS = 2048;
constexpr int SCALE_PAGES = 2048;  // pages whose scales are worked out at a time
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_UNROLL = 4;     // rows of a thread in a round
constexpr int KEY_CAP = 40960;     // weights that a block keeps in shared memory

struct Params {
  uint8_t* pages[2];     // k, v
  float* scale[2];       // 8-bit caches
  float* w;
  long long page_bytes, head_bytes, token_bytes;
  int num_pages, page_size, Hkv;
  const int *lens, *table;
  int table_stride, B, cap;
  int budget, recent;
  int* kept;      // [B][Hkv][budget]
  int* new_lens;  // [B]
  int2* src;      // workspace, [B][Hkv][budget]: page and slot of each kept token
  float* ratio;   // 8-bit caches, [2][B][Hkv][budget]: old scale / new scale
  int* first;     // [B][Hkv]: tokens in front that stay where they are
  int keys;       // weights that fit into the block's shared memory
  int row_pieces, slice_pieces, slices;  // 16-byte pieces of a row, and of a block's columns
  int* status;
};

// weights in the order of unsigned numbers; NaN above all, both zeros the same
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  if (w != w) return 0xffffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct SelectSmem {
  uint32_t hist[BINS];
  uint32_t part[SELECT_WARPS], part2[SELECT_WARPS];
  uint32_t bin, above;
  int lowest;  // first position that goes
};

template <bool F8>
__global__ void __launch_bounds__(SELECT_THREADS, 1) fa_evict_select_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) uint8_t raw[];
  SelectSmem& sm = *reinterpret_cast<SelectSmem*>(raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(raw + sizeof(SelectSmem));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
  launch_dependents();
  wait_previous_grid();
  const int told = p.lens[b], len = max(0, min(told, p.cap));
  const int* table = p.table + (size_t)b * p.table_stride;
  const size_t at0 = (size_t)blockIdx.x * p.budget;
  int* kept = p.kept + at0;
  if (tid == 0 && told > p.cap) atomicCAS(p.status, 0, FA_ERR_RANGE);
  if (len <= p.budget) {
    for (int j = tid; j < p.budget; j += SELECT_THREADS) kept[j] = j < len ? j : -1;
    if (tid == 0) p.first[blockIdx.x] = p.budget;
    return;
  }
  const int early = len - p.recent, need = p.budget - p.recent;  // 0 <= need < early
  auto load_key = [&](int i) -> uint32_t {
    const int page = table[(uint32_t)i / (uint32_t)p.page_size];
    if (page < 0 || page >= p.num_pages) {
      atomicCAS(p.status, 0, FA_ERR_RANGE);
      return 0;
    }
    return order_of(p.w[((size_t)page * p.Hkv + h) * p.page_size + (uint32_t)i % (uint32_t)p.page_size]);
  };
  const bool cached = early <= p.keys;
  if (cached) {
#pragma unroll 8
    for (int i = tid; i < early; i += SELECT_THREADS) keys[i] = load_key(i);
  }
  auto key_at = [&](int i) { return cached ? keys[i] : load_key(i); };
  // the need-th largest: its bits from the top, and how many of those equal to it stay
  uint32_t border = 0, left = (uint32_t)need;
  if (need > 0) {
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10, top = shift;
      shift -= bits;
      for (int i = tid; i < BINS; i += SELECT_THREADS) sm.hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int i = tid; i < early; i += SELECT_THREADS) {
        const uint32_t k = key_at(i);
        if (pass == 0 || (k >> top) == (border >> top)) atomicAdd(&sm.hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // thread: bins 2t and 2t + 1 from above; the bin in which the count from above passes `left`
      const uint32_t hi = sm.hist[BINS - 1 - 2 * tid], lo = sm.hist[BINS - 2 - 2 * tid];
      uint32_t incl = hi + lo;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) sm.part[warp] = incl;
      __syncthreads();
      uint32_t before = 0;
      for (int w = 0; w < warp; ++w) before += sm.part[w];
      const uint32_t up = before + incl - hi - lo;  // in bins above the thread's
      if (up < left && left <= up + hi + lo) {
        const bool first = left <= up + hi;
        sm.bin = BINS - 1 - 2 * tid - (first ? 0 : 1);
        sm.above = first ? up : up + hi;
      }
      __syncthreads();
      border |= sm.bin << shift;
      left -= sm.above;
    }
  }
  // counts of each warp's run of the early positions
  const int run = ((early + SELECT_WARPS - 1) / SELECT_WARPS + 31) & ~31;
  const int i0 = min(warp * run, early), i1 = min(i0 + run, early);
  uint32_t more = 0, same = 0;
  if (need > 0) {
#pragma unroll 4
    for (int i = i0; i < i1; i += 32) {
      const bool in = i + lane < i1;
      const uint32_t k = in ? key_at(i + lane) : 0u;
      more += __popc(__ballot_sync(0xffffffffu, in && k > border));
      same += __popc(__ballot_sync(0xffffffffu, in && k == border));
    }
  }
  __syncthreads();
  if (lane == 0) {
    sm.part[warp] = more;
    sm.part2[warp] = same;
  }
  if (tid == 0) sm.lowest = early;
  __syncthreads();
  uint32_t place = 0, ties = 0;
  for (int w = 0; w < warp; ++w) {
    place += sm.part[w] + min(sm.part2[w], left - min(ties, left));
    ties += sm.part2[w];
  }
  int2* src = p.src + at0;
  auto keep = [&](int j, int i) {
    kept[j] = i;
    const int page = table[(uint32_t)i / (uint32_t)p.page_size];
    src[j] = make_int2(page, (int)((uint32_t)i % (uint32_t)p.page_size));
  };
  int lowest = early;
#pragma unroll 2
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t k = in && need > 0 ? key_at(i + lane) : 0u;
    const bool is_same = in && need > 0 && k == border;
    const uint32_t tied = __ballot_sync(0xffffffffu, is_same), below = (1u << lane) - 1u;
    const bool stays = in && need > 0 && (k > border || (is_same && ties + __popc(tied & below) < left));
    const uint32_t all = __ballot_sync(0xffffffffu, stays);
    if (stays) keep((int)(place + __popc(all & below)), i + lane);
    else if (in) lowest = min(lowest, i + lane);
    place += __popc(all);
    ties += __popc(tied);
  }
  for (int r = tid; r < p.recent; r += SELECT_THREADS) keep(need + r, early + r);
  atomicMin(&sm.lowest, lowest);
  __syncthreads();  // (with the block's own global writes)
  if (tid == 0) p.first[blockIdx.x] = F8 ? sm.lowest / p.page_size * p.page_size : sm.lowest;
  if constexpr (F8) {
    // New scales, some pages at a time; the sources of later pages lie in later pages, whose scales still stand.
    uint32_t* tops = keys;  // [2][SCALE_PAGES], positive numbers in the order of their bits
    const int group = p.page_size >= SELECT_THREADS * 8 ? 1 : min(SCALE_PAGES, SELECT_THREADS * 8 / p.page_size);
    const size_t plane = (size_t)p.B * p.Hkv * p.budget;
    const int pages = (p.budget + p.page_size - 1) / p.page_size;
    for (int g0 = 0; g0 < pages; g0 += group) {
      const int n = min(group, pages - g0), j0 = g0 * p.page_size;
      const int j1 = (int)min((long long)p.budget, (long long)(g0 + n) * p.page_size);
      __syncthreads();
      for (int i = tid; i < 2 * SCALE_PAGES; i += SELECT_THREADS) tops[i] = 0;
      __syncthreads();
      auto scales_of = [&](int j, float (&s)[2]) {
        const int page = src[j].x;
        const bool ok = page >= 0 && page < p.num_pages;
#pragma unroll
        for (int x = 0; x < 2; ++x) s[x] = ok ? p.scale[x][(size_t)page * p.Hkv + h] : 0.f;
      };
#pragma unroll 4
      for (int j = j0 + tid; j < j1; j += SELECT_THREADS) {
        float s[2];
        scales_of(j, s);
        const int at = (j - j0) / p.page_size;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (s[x] > 0.f) atomicMax(&tops[x * SCALE_PAGES + at], __float_as_uint(s[x]));
      }
      __syncthreads();
#pragma unroll 4
      for (int j = j0 + tid; j < j1; j += SELECT_THREADS) {
        float s[2];
        scales_of(j, s);
        const int at = (j - j0) / p.page_size;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float top = __uint_as_float(tops[x * SCALE_PAGES + at]);
          p.ratio[x * plane + at0 + j] = top > 0.f ? s[x] / top : 1.f;
        }
      }
      __syncthreads();
      for (int i = tid; i < 2 * n; i += SELECT_THREADS) {
        const int x = i >= n, at = x ? i - n : i, page = table[g0 + at];
        const uint32_t top = tops[x * SCALE_PAGES + at];
        if (page >= 0 && page < p.num_pages && top) p.scale[x][(size_t)page * p.Hkv + h] = __uint_as_float(top);
      }
    }
  }
}

// Blocks of a (sequence, key head): `slices` of k, of v, and one for its weights.
template <bool F8>
__global__ void __launch_bounds__(MOVE_THREADS) fa_evict_move_kernel(const __grid_constant__ Params p) {
  const int per = 2 * p.slices + 1;
  const int bh = blockIdx.x / per, unit = blockIdx.x - bh * per;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  launch_dependents();
  wait_previous_grid();
  // here, not beside the selection: new_lens may be lens, which that reads in every block of the sequence
  if (h == 0 && unit == 0 && threadIdx.x == 0) p.new_lens[b] = min(max(0, min(p.lens[b], p.cap)), p.budget);
  const int first = p.first[bh];
  if (first >= p.budget) return;
  const int* table = p.table + (size_t)b * p.table_stride;
  const size_t at0 = (size_t)bh * p.budget;
  const int2* src = p.src + at0;
  auto fine = [&](int page) { return page >= 0 && page < p.num_pages; };
  constexpr int U = MOVE_UNROLL;
  if (unit == 2 * p.slices) {
    float* w = p.w + (size_t)h * p.page_size;
    const size_t stride = (size_t)p.Hkv * p.page_size;
    float cur[U], nxt[U];
    auto load = [&](int j0, float (&v)[U]) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int j = j0 + i * MOVE_THREADS + (int)threadIdx.x;
        if (j >= p.budget) continue;
        const int2 s = src[j];
        v[i] = fine(s.x) ? w[(size_t)s.x * stride + s.y] : 0.f;
      }
    };
    load(first, cur);
    for (int j0 = first; j0 < p.budget; j0 += U * MOVE_THREADS) {
      load(j0 + U * MOVE_THREADS, nxt);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int j = j0 + i * MOVE_THREADS + (int)threadIdx.x;
        if (j < p.budget) {
          const int page = table[(uint32_t)j / (uint32_t)p.page_size];
          if (fine(page)) w[(size_t)page * stride + (uint32_t)j % (uint32_t)p.page_size] = cur[i];
        }
        cur[i] = nxt[i];
      }
    }
    return;
  }
  const int set = unit >= p.slices, slice = set ? unit - p.slices : unit;
  const int rows = MOVE_THREADS / p.slice_pieces, row = (int)threadIdx.x / p.slice_pieces;
  const int piece = slice * p.slice_pieces + (int)threadIdx.x - row * p.slice_pieces;
  uint8_t* base = p.pages[set] + (long long)h * p.head_bytes + piece * 16;
  const float* ratios = F8 ? p.ratio + (set ? (size_t)p.B * p.Hkv * p.budget : 0) + at0 : nullptr;
  const int round = rows * U;
  uint4 cur[U], nxt[U];
  float cur_r[U], nxt_r[U];
  auto load = [&](int j0, uint4 (&v)[U], float (&r)[U]) {
    int2 s[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * rows + row;
      s[i] = j < p.budget ? src[j] : make_int2(-1, 0);
      r[i] = F8 && j < p.budget ? ratios[j] : 1.f;
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (fine(s[i].x)) v[i] = *reinterpret_cast<const uint4*>(base + (long long)s[i].x * p.page_bytes + (long long)s[i].y * p.token_bytes);
  };
  load(first, cur, cur_r);
  for (int j0 = first; j0 < p.budget; j0 += round) {
    load(j0 + round, nxt, nxt_r);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * rows + row;
      if (j < p.budget) {
        const int page = table[(uint32_t)j / (uint32_t)p.page_size];
        if (F8 && cur_r[i] != 1.f) {
          uint32_t* c = reinterpret_cast<uint32_t*>(&cur[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t lo, hi;
            float f[4];
            unpack4_e4m3(c[e], lo, hi);
            unpack2<false>(lo, f[0], f[1]);
            unpack2<false>(hi, f[2], f[3]);
            c[e] = pack4_e4m3(f[0] * cur_r[i], f[1] * cur_r[i], f[2] * cur_r[i], f[3] * cur_r[i]);
          }
        }
        if (fine(page) && fine(src[j].x))
          *reinterpret_cast<uint4*>(base + (long long)page * p.page_bytes +
                                    (long long)((uint32_t)j % (uint32_t)p.page_size) * p.token_bytes) = cur[i];
      }
      cur[i] = nxt[i];
      cur_r[i] = nxt_r[i];
    }
  }
}

}  // namespace evict
}  // namespace fa
