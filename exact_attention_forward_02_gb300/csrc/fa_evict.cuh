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
// its loads and its stores, makes the move safe in place.
//
// 8 sequences of 8 heads cut from 30 thousand tokens and more to 16384, d 128, 8 bits: 56 us for the selection, whose 64
// blocks have 64 SMs and issue in 56 % of their slots, and 113 for the move, 4.7 TB/s: with narrow columns each
// request of a warp touches up to 16 rows. Wider ones leave too few blocks (64 bytes: 191 us in all for 170), copies
// through shared memory, more rounds ahead, gained nothing (172 to 201). One sequence: 16 us, latency.
#pragma once

#include "fa_rope.cuh"

namespace fa {
namespace evict {

constexpr int SELECT_THREADS = 1024, SELECT_WARPS = 32;
constexpr int BINS = 2048;
constexpr int SCALE_PAGES = 2048;  // pages whose scales are worked out at a time
constexpr int MOVE_THREADS = 256;
__host__ __device__ constexpr int move_unroll(bool f8) { return f8 ? 2 : 4; }  // rows of a thread in a round
constexpr int KEY_CAP = 40960;     // weights that a block keeps in shared memory

struct Params {
  uint8_t* pages[2];     // k, v
  float* scale[2];       // 8-bit caches
  float* w;
  long long page_bytes, head_bytes, token_bytes;
  int num_pages, page_size, Hkv;
  int page_shift;        // log2 of the page size, -1 where that is none
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

// page and slot of position j
__device__ __forceinline__ int2 place_of(const Params& p, int j) {
  const int at = p.page_shift >= 0 ? j >> p.page_shift : (int)((uint32_t)j / (uint32_t)p.page_size);
  return make_int2(at, j - at * p.page_size);
}

// four codes under a smaller scale. In fp16 by a power of two, exactly: below 2^-24, where fp16 cuts off, nothing
// reaches half of E4M3's least number (2^-10).
__device__ __forceinline__ uint32_t codes_times(uint32_t c, float r, bool power) {
  uint32_t lo, hi;
  unpack4_e4m3(c, lo, hi);
  if (power) {
    const uint32_t r2 = pack2<false>(r, r);
    asm("{\n\t.reg .b32 a, b;\n\t.reg .b16 x, y;\n\t"
        "mul.rn.f16x2 a, %1, %3;\n\tmul.rn.f16x2 b, %2, %3;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 x, a;\n\tcvt.rn.satfinite.e4m3x2.f16x2 y, b;\n\t"
        "mov.b32 %0, {x, y};\n\t}"
        : "=r"(c)
        : "r"(lo), "r"(hi), "r"(r2));
    return c;
  }
  float f[4];
  unpack2<false>(lo, f[0], f[1]);
  unpack2<false>(hi, f[2], f[3]);
  return pack4_e4m3(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
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
  // (straight code: the loads of several positions are on their way together)
  bool bad = false;
  auto load_key = [&](int i) -> uint32_t {
    const int2 at = place_of(p, i);
    const int page = table[at.x];
    const bool fine = page >= 0 && page < p.num_pages;
    const float w = fine ? p.w[((size_t)page * p.Hkv + h) * p.page_size + at.y] : 0.f;
    bad |= !fine;
    return fine ? order_of(w) : 0u;
  };
  const bool cached = early <= p.keys;
  if (cached) {
    constexpr int AT_ONCE = 8;
#pragma unroll 1
    for (int i0 = tid; i0 < early; i0 += AT_ONCE * SELECT_THREADS) {
      uint32_t k[AT_ONCE];
#pragma unroll
      for (int y = 0; y < AT_ONCE; ++y) k[y] = load_key(min(i0 + y * SELECT_THREADS, early - 1));
#pragma unroll
      for (int y = 0; y < AT_ONCE; ++y)
        if (i0 + y * SELECT_THREADS < early) keys[i0 + y * SELECT_THREADS] = k[y];
    }
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
      const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? sm.part[lane] : 0u);
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
  uint32_t ties = __reduce_add_sync(0xffffffffu, lane < warp ? sm.part2[lane] : 0u);
  uint32_t place = __reduce_add_sync(0xffffffffu, lane < warp ? sm.part[lane] : 0u) + min(ties, left);
  int2* src = p.src + at0;
  auto keep = [&](int j, int i, int page) {
    if (!in_bounds(p, j >= 0 && j < p.budget && i >= j && i < len)) return;
    kept[j] = i;
    src[j] = make_int2(page, place_of(p, i).y);
  };
  int lowest = early;
  auto page_of = [&](int i) { return i < i1 ? table[place_of(p, i).x] : -1; };
  int ahead[4];  // the pages of the next 128 positions
#pragma unroll
  for (int y = 0; y < 4; ++y) ahead[y] = page_of(i0 + y * 32 + lane);
#pragma unroll 1
  for (int i = i0; i < i1; i += 32) {
    const int page = ahead[0];
    ahead[0] = ahead[1], ahead[1] = ahead[2], ahead[2] = ahead[3];
    ahead[3] = page_of(i + 128 + lane);
    const bool in = i + lane < i1;
    const uint32_t k = in && need > 0 ? key_at(i + lane) : 0u;
    const bool is_same = in && need > 0 && k == border;
    const uint32_t tied = __ballot_sync(0xffffffffu, is_same), below = (1u << lane) - 1u;
    const bool stays = in && need > 0 && (k > border || (is_same && ties + __popc(tied & below) < left));
    const uint32_t all = __ballot_sync(0xffffffffu, stays);
    if (stays) keep((int)(place + __popc(all & below)), i + lane, page);
    else if (in) lowest = min(lowest, i + lane);
    place += __popc(all);
    ties += __popc(tied);
  }
  for (int r = tid; r < p.recent; r += SELECT_THREADS) {
    const int page = table[place_of(p, early + r).x];
    bad |= page < 0 || page >= p.num_pages;
    keep(need + r, early + r, page);
  }
  if (need == 0 && !cached)  // no weight has been asked for
    for (int e = tid; e < place_of(p, early).x; e += SELECT_THREADS) bad |= table[e] < 0 || table[e] >= p.num_pages;
  atomicMin(&sm.lowest, lowest);
  __syncthreads();  // (with the block's own global writes)
  if (bad) atomicCAS(p.status, 0, FA_ERR_RANGE);
  if (tid == 0) p.first[blockIdx.x] = F8 ? sm.lowest / p.page_size * p.page_size : sm.lowest;
  if constexpr (F8) {
    // New scales, some pages at a time; the sources of later pages lie in later pages, whose scales still stand.
    // [2][SCALE_PAGES], numbers that are not negative in the order of their bits, + 1; 0: no token came from a page
    uint32_t* tops = keys;
    constexpr int AT_ONCE = 8, CHUNK = AT_ONCE * SELECT_THREADS;
    const int group = p.page_size >= CHUNK ? 1 : min(SCALE_PAGES, CHUNK / p.page_size);
    const size_t plane = (size_t)p.B * p.Hkv * p.budget;
    const int pages = (p.budget + p.page_size - 1) / p.page_size;
    for (int g0 = 0; g0 < pages; g0 += group) {
      const int n = min(group, pages - g0), j0 = g0 * p.page_size;
      const int j1 = (int)min((long long)p.budget, (long long)(g0 + n) * p.page_size);
      float s[AT_ONCE][2];
      auto fetch = [&](int c0) {  // the scales that a thread's tokens come from
        int from[AT_ONCE];
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
          const int j = c0 + y * SELECT_THREADS + tid;
          from[y] = j < j1 ? src[j].x : -1;
        }
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
          const bool ok = from[y] >= 0 && from[y] < p.num_pages;
#pragma unroll
          for (int x = 0; x < 2; ++x) s[y][x] = ok ? p.scale[x][(size_t)from[y] * p.Hkv + h] : -1.f;
        }
      };
      __syncthreads();
      for (int i = tid; i < 2 * SCALE_PAGES; i += SELECT_THREADS) tops[i] = 0;
      __syncthreads();
#pragma unroll 1
      for (int c0 = j0; c0 < j1; c0 += CHUNK) {  // more than one chunk only where a page is larger
        fetch(c0);
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
          const int at = place_of(p, c0 + y * SELECT_THREADS + tid - j0).x;
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (s[y][x] >= 0.f) atomicMax(&tops[x * SCALE_PAGES + at], s[y][x] > 0.f ? __float_as_uint(s[y][x]) + 1u : 1u);
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int c0 = j0; c0 < j1; c0 += CHUNK) {
        if (j1 - j0 > CHUNK) fetch(c0);
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
          const int j = c0 + y * SELECT_THREADS + tid;
          if (j >= j1) break;
          const int at = place_of(p, j - j0).x;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float top = __uint_as_float(max(tops[x * SCALE_PAGES + at], 1u) - 1u);
            p.ratio[x * plane + at0 + j] = top > 0.f ? s[y][x] / top : 1.f;
          }
        }
      }
      __syncthreads();
      for (int i = tid; i < 2 * n; i += SELECT_THREADS) {
        const int x = i >= n, at = x ? i - n : i, page = table[g0 + at];
        const uint32_t top = tops[x * SCALE_PAGES + at];
        if (page >= 0 && page < p.num_pages && top) p.scale[x][(size_t)page * p.Hkv + h] = __uint_as_float(top - 1u);
      }
    }
  }
}

// Blocks of a (sequence, key head): `slices` of k, of v, and one for its weights.
template <bool F8>
__global__ void __launch_bounds__(MOVE_THREADS, 4) fa_evict_move_kernel(const __grid_constant__ Params p) {
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
  constexpr int U = move_unroll(F8);
  // Three rounds at once: one's stores, the next one's rows on their way, and where those after it come from.
  const bool weights = unit == 2 * p.slices;
  const int set = unit >= p.slices, slice = set ? unit - p.slices : unit;
  const int rows = weights ? MOVE_THREADS : MOVE_THREADS / p.slice_pieces;
  const int row = weights ? (int)threadIdx.x : (int)threadIdx.x / p.slice_pieces;
  const int round = rows * U;
  const float* ratios = F8 && !weights ? p.ratio + (set ? (size_t)p.B * p.Hkv * p.budget : 0) + at0 : nullptr;
  auto sources = [&](int j0, int2 (&s)[U]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * rows + row;
      s[i] = j < p.budget ? src[j] : make_int2(-1, 0);
    }
  };
  auto walk = [&](auto zero, auto load, auto store) {
    decltype(zero) cur[U], nxt[U];
    float cur_r[U], nxt_r[U];
    int2 s[U];
    uint32_t cur_ok = 0, nxt_ok = 0;
    auto rows_of = [&](int j0, decltype(cur)& v, float (&r)[U], uint32_t& ok) {
      ok = 0;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (s[i].x < 0 || s[i].x >= p.num_pages || !in_bounds(p, s[i].y >= 0 && s[i].y < p.page_size)) continue;
        ok |= 1u << i;
        v[i] = load(s[i]);
        r[i] = F8 && !weights ? ratios[j0 + i * rows + row] : 1.f;
      }
    };
    sources(first, s);
    rows_of(first, cur, cur_r, cur_ok);
    sources(first + round, s);
#pragma unroll 1
    for (int j0 = first; j0 < p.budget; j0 += round) {
      rows_of(j0 + round, nxt, nxt_r, nxt_ok);
      sources(j0 + 2 * round, s);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (cur_ok >> i & 1u) {
          const int2 at = place_of(p, j0 + i * rows + row);
          const int page = table[at.x];
          if (page >= 0 && page < p.num_pages && in_bounds(p, at.x < p.table_stride && at.y >= 0 && at.y < p.page_size))
            store(make_int2(page, at.y), cur[i], cur_r[i]);
        }
        cur[i] = nxt[i];
        cur_r[i] = nxt_r[i];
      }
      cur_ok = nxt_ok;
    }
  };
  if (weights) {
    float* w = p.w + (size_t)h * p.page_size;
    const size_t stride = (size_t)p.Hkv * p.page_size;
    walk(0.f, [&](int2 s) { return w[(size_t)s.x * stride + s.y]; },
         [&](int2 to, float v, float) { w[(size_t)to.x * stride + to.y] = v; });
    return;
  }
  const int piece = slice * p.slice_pieces + (int)threadIdx.x - row * p.slice_pieces;
  uint8_t* base = p.pages[set] + (long long)h * p.head_bytes + piece * 16;
  auto at = [&](int2 s) {
    return reinterpret_cast<uint4*>(base + (long long)s.x * p.page_bytes + (long long)s.y * p.token_bytes);
  };
  walk(uint4{}, [&](int2 s) { return *at(s); },
       [&](int2 to, uint4 v, float r) {
         if (F8 && r != 1.f) {
           const bool power = (__float_as_uint(r) & 0x7fffffu) == 0;
           v = make_uint4(codes_times(v.x, r, power), codes_times(v.y, r, power), codes_times(v.z, r, power),
                          codes_times(v.w, r, power));
         }
         *at(to) = v;
       });
}

}  // namespace evict
}  // namespace fa
