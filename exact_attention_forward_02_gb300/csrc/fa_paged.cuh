// fa_paged.cuh -- attention of new tokens over a paged cache of keys and values (forward).
// Included by fa_decoder.cu.
//
//   O_i = sum_j softmax_j(scale <q_i, k_j>) v_j,   L_i = ln sum_j exp(scale <q_i, k_j>)
// over the keys j < len of row i's sequence (with a causal mask, up to its own position), by the
// recurrence of the online softmax over tiles of 128 keys (m: running maximum, l: running sum).
//
// Rows. The G query heads that share a key head are rows of one tile: row r of a tile of T tokens
// is token r / G, head r % G, so that a key is loaded once for all of them (for single tokens
// this is what makes G rows of work from one pass over the cache).
//
// Work. An item is (sequence, key head, block of tokens); its keys are cut into tiles of 128,
// and a unit is one (item, tile). The lengths are device data, so every block adds up the units
// of all sequences by itself (a closed form per sequence), and block c of Ge takes the units
// [c W / Ge, (c+1) W / Ge) of the W in order. An item that lies in several blocks' ranges leaves
// partial states (m, l, O~) in the workspace; fa_paged_combine_kernel joins them, in the order of
// the blocks. Nothing in the main kernel waits on another block.
//
// Two forms of the kernel, of 12 warps (8: loads of Q and K, 11: loads of V, 9: MMA issuer, 10:
// walks the block's range and hands the others their items through a ring in shared memory, a few
// ahead, so that nobody waits for the lengths of the next sequence; 0-7: two softmax warpgroups,
// thread = row = TMEM lane):
//   PAIR   an item is two tiles of 128 rows, one per warpgroup, over the same keys: long chunks,
//          bound by the tensor cores.
//   SPLIT  an item is one tile; the warpgroups take the even and the odd key tiles, each with its
//          own (m, l, O~). Its rows stand REP times in the tile (REP = 4 for up to 32 rows): copy
//          a covers keys [a 128/REP, (a+1) 128/REP) of each key tile only, with its own (m, l, O~)
//          and zeros in P elsewhere. So each warp reads 128/REP scores of each row instead of one
//          warp reading 128; nothing is exchanged before the item's end. Single tokens and
//          drafts: bound by HBM; the tensor cores run mostly empty and still hide behind the
//          loads (1024 cycles of products per 64 KB of keys and values, which take 2900 at this
//          SM's share of the bandwidth).
#pragma once

#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include "fa_rope.cuh"

namespace fa {
namespace paged {

constexpr int BM = 128, BN = 128;
constexpr int NUM_WARPS = 12, NUM_THREADS = NUM_WARPS * 32;
constexpr int WARP_LOAD = 8, WARP_MMA = 9, WARP_WALK = 10, WARP_LOAD_V = 11;
constexpr int ITEM_SLOTS = 4;
constexpr int ITEM_READERS = 11;  // warps that read an item: two loading, MMA, 8 softmax
// 2*128*200 + 128*104 = 64512 = 384*168 registers, the launch's budget
constexpr uint32_t REGS_SOFTMAX = 200, REGS_OTHER = 104;
constexpr uint32_t TMEM_COLS = 512, TMEM_S0 = 0, TMEM_O0 = 256;  // S0 | S1 | O0 | O1
constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units, as in the dense kernel
constexpr int SMEM_LIMIT = 232448;
constexpr int MAX_SLOTS = 8;
constexpr int COMBINE_THREADS = 256;

struct Params {
  HeadsDev o;
  float* L;
  int num_pages, page_size, box_keys;  // box_keys: keys per TMA box, min(page_size, 128)
  int Hkv, G, tpt;                     // tpt: tokens per tile, (128 / REP) / G
  const int *cu, *lens, *table;
  int table_stride, B, T, causal;
  float c;  // scale * log2(e)
  unsigned long long wait_limit_ns;
  int* status;
  int* records;  // [block][8]: the item that begins in a block's range and ends in another's
  float* parts;  // [block][2][rows]: D floats of O~ per row, then [rows][2] of (m, l)
};

__host__ __device__ constexpr int part_floats(int d, int rows) { return rows * (d + 2); }

// One block's part of one item.
struct Item {
  int b, h, tok0, nt;   // sequence, key head, first row of q, tokens
  int len, vis0;        // cached tokens; keys that the item's first token sees (causal)
  int j0, n, ntot;      // key tiles [j0, j0 + n) of ntot; n = 0: no more items
  int n0;               // PAIR: of the n, those that reach the first tile's rows (at least 1)
  int slot;             // place of its partial state: 0 = first piece of the block's range
};

struct Barriers {
  uint64_t q_full, q_empty;
  uint64_t kv_full[MAX_SLOTS], kv_release[MAX_SLOTS];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t mma_drain, epi;
  uint64_t item_full[ITEM_SLOTS], item_empty[ITEM_SLOTS];
  Item items[ITEM_SLOTS];
  long long warp_units[NUM_WARPS];
  long long rem;  // units of the first sequence before this block's range
  int first_b, first_h, first_q, first_j;
  uint32_t tmem_base;
  int abort_flag;
};

template <int D, bool SPLIT>
struct Layout {
  static constexpr int TILE_BYTES = BM * D * 2;
  static constexpr int CHUNK_BYTES = BM * 128, CHUNKS = D / 64;
  static constexpr int Q_TILES = SPLIT ? 1 : 2;
  static constexpr int STAGE_BYTES = SPLIT ? BM * D * 4 : 0;  // one fp32 tile of O~
  static constexpr int HEAD_BYTES = 1024 + 1024;              // barriers, alignment
  static constexpr int FIT = (SMEM_LIMIT - Q_TILES * TILE_BYTES - STAGE_BYTES - HEAD_BYTES) / TILE_BYTES;
  static constexpr int KV_SLOTS = FIT > MAX_SLOTS ? MAX_SLOTS : FIT;
  static constexpr int OFF_Q = 0, OFF_KV = Q_TILES * TILE_BYTES;
  static constexpr int OFF_STAGE = OFF_KV + KV_SLOTS * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_STAGE + STAGE_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + HEAD_BYTES;
  static_assert(sizeof(Barriers) <= 1024 && KV_SLOTS >= 4 && SMEM_BYTES <= SMEM_LIMIT, "shared memory budget");
};

// ----------------------------------------------------------------------------- waits
// Bounded: a wait past the limit records FA_ERR_TIMEOUT and stops every role of the block.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, const Params& p) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > p.wait_limit_ns) {
      atomicCAS(p.status, 0, FA_ERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, const Params& p) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, abort_flag, p);
}
// on the way out after an abort: ignores the flag, still bounded
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, const Params& p) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > p.wait_limit_ns) {
      atomicCAS(p.status, 0, FA_ERR_TIMEOUT);
      return;
    }
}

// ----------------------------------------------------------------------------- schedule
struct Seq {
  int t0, n, len, nq;  // first row of q, new tokens, tokens in the cache, blocks of tokens
};

// Sequence b as the kernels see it: a range of rows outside [0, T] counts as empty, a length
// past the table's width is cut to it; `report` records either.
template <int TPT_MUL>
__device__ __forceinline__ Seq load_seq(const Params& p, int b, bool report) {
  Seq s;
  s.t0 = p.cu[b];
  const long long n = (long long)p.cu[b + 1] - s.t0;
  const long long cap = (long long)p.table_stride * p.page_size;
  const int len = p.lens[b];
  const bool rows_ok = s.t0 >= 0 && n >= 0 && s.t0 + n <= p.T;
  s.n = rows_ok ? (int)n : 0;
  s.len = len < 0 ? 0 : (int)(len > cap ? cap : len);
  const int tpi = p.tpt * TPT_MUL;
  s.nq = (s.n + tpi - 1) / tpi;
  if (report && (!rows_ok || (s.n && len > cap))) atomicCAS(p.status, 0, FA_ERR_RANGE);
  return s;
}

// key tiles of block q of a sequence (at least one, so that its rows are written)
__device__ __forceinline__ int tiles_of(const Params& p, const Seq& s, int q, int tpi) {
  long long vis = s.len;
  if (p.causal) {
    const long long end = (long long)(q + 1) * tpi;
    vis = (long long)s.len - s.n + (end < s.n ? end : s.n);
  }
  return vis <= 0 ? 1 : (int)((vis + BN - 1) / BN);
}

// sum over i < n of floor((a i + b) / m), for a, b >= 0 (by Euclid's steps on (a, m))
__device__ __forceinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (true) {
    if (a >= m) s += (n - 1) * n / 2 * (a / m), a %= m;
    if (b >= m) s += n * (b / m), b %= m;
    const long long y = a * n + b;
    if (y < m) return s;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
}

// key tiles of the blocks before q (q <= nq - 1: whole blocks only)
__device__ __forceinline__ long long tiles_before(const Params& p, const Seq& s, int q, int tpi) {
  if (q == 0) return 0;
  if (!p.causal) return (long long)q * tiles_of(p, s, 0, tpi);
  // block i ends at key ctx + (i + 1) tpi; the first k0 of them reach key 128 at most: one tile
  const long long ctx = (long long)s.len - s.n;
  long long k0 = BN - ctx < 0 ? 0 : (BN - ctx) / tpi;
  if (k0 > q) k0 = q;
  return k0 + (q > k0 ? floor_sum(q - k0, BN, tpi, ctx + (k0 + 1) * tpi + BN - 1) : 0);
}
__device__ __forceinline__ long long tiles_total(const Params& p, const Seq& s, int tpi) {
  return s.nq ? tiles_before(p, s, s.nq - 1, tpi) + tiles_of(p, s, s.nq - 1, tpi) : 0;
}

struct Range {
  long long W, u0, u1;
  int Ge;  // blocks that take part
};
__device__ __forceinline__ long long bound_of(long long c, const Range& r) { return c * r.W / r.Ge; }
__device__ __forceinline__ int owner_of(long long u, const Range& r) {
  long long c = u * r.Ge / r.W;
  while (c + 1 < r.Ge && bound_of(c + 1, r) <= u) ++c;
  return (int)c;
}

// Walks a block's range.
template <int TPT_MUL>
struct Walk {
  Seq s;
  int b, h, q, j;
  long long u;
  bool first;
  __device__ __forceinline__ void begin(const Params& p, const Range& r, const Barriers* bars) {
    b = bars->first_b;
    h = bars->first_h;
    q = bars->first_q;
    j = bars->first_j;
    u = r.u0;
    first = true;
    if (u < r.u1) s = load_seq<TPT_MUL>(p, b, false);
  }
  // `last`: the block that ends the item
  __device__ __forceinline__ bool next(const Params& p, const Range& r, Item& it, int& last) {
    if (u >= r.u1) return false;
    const int tpi = p.tpt * TPT_MUL;
    if (q == s.nq) {
      q = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          if (++b >= p.B) return false;
          s = load_seq<TPT_MUL>(p, b, false);
        } while (s.n == 0);
      }
    }
    it.b = b;
    it.h = h;
    it.tok0 = s.t0 + q * tpi;
    it.nt = min(tpi, s.n - q * tpi);
    it.len = s.len;
    it.vis0 = s.len - s.n + q * tpi + 1;
    it.ntot = tiles_of(p, s, q, tpi);
    it.j0 = j;
    const long long left = r.u1 - u;
    it.n = left < it.ntot - j ? (int)left : it.ntot - j;
    it.slot = first ? 0 : 1;
    it.n0 = it.n;
    if (TPT_MUL == 2 && p.causal) {
      const long long vis = (long long)it.vis0 + min(p.tpt, it.nt) - 1;
      const long long t = (vis <= 0 ? 1 : (vis + BN - 1) / BN) - j;
      it.n0 = t < 1 ? 1 : (t < it.n ? (int)t : it.n);
    }
    last = it.n == it.ntot ? (int)blockIdx.x : owner_of(u - j + it.ntot - 1, r);
    first = false;
    u += it.n;
    j = 0;
    ++q;
    return true;
  }
};

// The block's share of the units, and where it begins. All threads call this; it ends with a
// barrier.
template <int TPT_MUL, int MIN_UNITS>
__device__ __forceinline__ Range plan(const Params& p, Barriers* bars) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tpi = p.tpt * TPT_MUL;
  const int chunk = (p.B + NUM_THREADS - 1) / NUM_THREADS;
  const int b0 = min(tid * chunk, p.B), b1 = min(b0 + chunk, p.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += p.Hkv * tiles_total(p, load_seq<TPT_MUL>(p, b, blockIdx.x == 0), tpi);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) bars->warp_units[warp] = incl;
  __syncthreads();
  long long before = incl - mine;
  Range r;
  r.W = 0;
#pragma unroll
  for (int w = 0; w < NUM_WARPS; ++w) {
    if (w < warp) before += bars->warp_units[w];
    r.W += bars->warp_units[w];
  }
  const long long most = (r.W + MIN_UNITS - 1) / MIN_UNITS;
  r.Ge = most < (long long)gridDim.x ? (int)most : (int)gridDim.x;
  r.u0 = r.u1 = 0;
  if ((int)blockIdx.x < r.Ge) {
    r.u0 = bound_of(blockIdx.x, r);
    r.u1 = bound_of(blockIdx.x + 1, r);
  }
  if (r.u0 < r.u1 && before <= r.u0 && r.u0 < before + mine) {
    for (int b = b0; b < b1; ++b) {
      const long long x = p.Hkv * tiles_total(p, load_seq<TPT_MUL>(p, b, false), tpi);
      if (r.u0 < before + x) {
        bars->first_b = b;
        bars->rem = r.u0 - before;
        break;
      }
      before += x;
    }
  }
  __syncthreads();
  if (warp == 0 && r.u0 < r.u1) {
    const Seq s = load_seq<TPT_MUL>(p, bars->first_b, false);
    const long long head = tiles_total(p, s, tpi);
    const int h = (int)(bars->rem / head);
    const long long rem = bars->rem - h * head;
    // the last block q with tiles_before(q) <= rem: 32 candidates at a time
    int lo = 0, n = s.nq;
    while (n > 1) {
      const int step = (n + 31) / 32, cand = lo + lane * step;
      const bool le = lane * step < n && tiles_before(p, s, cand, tpi) <= rem;
      const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;  // candidate 0 always holds
      lo += k * step;
      n = min(step, n - k * step);
    }
    if (lane == 0) {
      bars->first_h = h;
      bars->first_q = lo;
      bars->first_j = (int)(rem - tiles_before(p, s, lo, tpi));
    }
  }
  __syncthreads();
  return r;
}

// ----------------------------------------------------------------------------- kernel
template <int D, bool BF16, bool SPLIT, int REP>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    fa_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  static_assert(SPLIT || REP == 1, "copies of rows belong to the SPLIT form");
  using LY = Layout<D, SPLIT>;
  constexpr int TPT_MUL = SPLIT ? 1 : 2;
  constexpr int ROWS = SPLIT ? BM / REP : 2 * BM;  // rows of an item's partial state
  constexpr int CW = BN / REP;                     // keys of a tile that one row copy covers
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Barriers* bars = reinterpret_cast<Barriers*>(smem + LY::OFF_BAR);
  const uint32_t sQ = smem_u32(smem + LY::OFF_Q), sKV = smem_u32(smem + LY::OFF_KV);
  const uint32_t sStage = smem_u32(smem + LY::OFF_STAGE);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), 1);
    for (int s = 0; s < LY::KV_SLOTS; ++s) {
      mbar_init(smem_u32(&bars->kv_full[s]), 1);
      mbar_init(smem_u32(&bars->kv_release[s]), 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_u32(&bars->s_full[g]), 1);
      mbar_init(smem_u32(&bars->p_full[g]), 4);
      mbar_init(smem_u32(&bars->o_done[g]), 1);
    }
    mbar_init(smem_u32(&bars->mma_drain), 1);
    mbar_init(smem_u32(&bars->epi), 8);
    for (int s = 0; s < ITEM_SLOTS; ++s) {
      mbar_init(smem_u32(&bars->item_full[s]), 1);
      mbar_init(smem_u32(&bars->item_empty[s]), ITEM_READERS);
    }
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == WARP_LOAD && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(&bars->tmem_base), TMEM_COLS);
    tmem_relinquish();
  }
  launch_dependents();
  tc_fence_before();
  const Range range = plan<TPT_MUL, SPLIT ? 2 : 1>(p, bars);
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // Items in order: the reader's place in the ring, and the item there (nullptr: the wait gave up).
  uint32_t n_item = 0;
  auto item_next = [&]() -> const Item* {
    const uint32_t s = n_item % ITEM_SLOTS;
    const bool w = wait_bar(smem_u32(&bars->item_full[s]), (n_item / ITEM_SLOTS) & 1u, abort_flag, p);
    return __all_sync(0xffffffffu, w) ? &bars->items[s] : nullptr;
  };
  auto item_done = [&]() {  // this warp needs nothing more of the item
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[n_item % ITEM_SLOTS]));
    ++n_item;
  };

  if (warp >= WARP_LOAD) {
    regs_dec<REGS_OTHER>();
    // Loads are numbered over the block's pieces in the order of their use; load i goes to slot
    // i mod KV_SLOTS. PAIR: K0 V0 K1 V1 ...; unit u = {V of tile u-1, K of tile u} is released at
    // once. SPLIT: K0 K1 V0 K2 V1 K3 ...; every load is released by itself.
    if (warp == WARP_LOAD || warp == WARP_LOAD_V) {
      // ======================================================================= producers
      // All 32 lanes: a tile's boxes (pages, and 64-column halves) are issued side by side. A box
      // costs its warp about 100 cycles whatever its size, so K and V have a warp each.
      const bool is_v = warp == WARP_LOAD_V;
      const CUtensorMap* tm = is_v ? &tmV : &tmK;
      const int boxes = BN / p.box_keys;                    // page boxes of one 64-column chunk
      const int tiles_per_page = p.page_size > BN ? p.page_size / BN : 1;
      const int my_box = lane % boxes, my_chunk = lane / boxes;
      const bool issues = my_chunk < LY::CHUNKS;
      const uint32_t box_bytes = (uint32_t)p.box_keys * 128u;
      const uint32_t box_off = (uint32_t)my_chunk * LY::CHUNK_BYTES + (uint32_t)my_box * box_bytes;
      uint32_t ld0 = 0, q_ph = 0, issued_mask = 0, last_par = 0;
      bool ok = true, q_issued = false;
      while (ok) {
        const Item* src = item_next();
        if (!(ok = src != nullptr)) break;
        const Item it = *src;
        item_done();
        if (it.n == 0) break;
        // 32 entries of the sequence's table at a time, one per lane; the next 32 are on their way
        const int* table = p.table + (size_t)it.b * p.table_stride;
        auto entries = [&](int window) -> int {
          const int e = window * 32 + lane;
          if ((long long)e * p.page_size >= it.len) return -1;  // holds no key of the sequence
          const int page = table[e];
          if (page >= 0 && page < p.num_pages) return page;
          atomicCAS(p.status, 0, FA_ERR_RANGE);
          return p.num_pages;  // reads as zeros
        };
        const int first = it.j0 / tiles_per_page * (p.page_size > BN ? 1 : boxes);
        int window = first / 32, held = entries(window), next = entries(window + 1);
        for (int i = 0; i < it.n; ++i) {
          const int j = it.j0 + i;
          const int e0 = p.page_size > BN ? j / tiles_per_page : j * boxes;  // the tile's first entry
          if (e0 / 32 != window) {  // 32 is a multiple of a tile's entries
            window = e0 / 32;
            held = next;
            next = entries(window + 1);
          }
          const int page = __shfl_sync(0xffffffffu, held, (e0 + my_box) % 32);
          const uint32_t ld = ld0 + (SPLIT ? (is_v ? 2 + i + min(i, it.n - 2) : i < 2 ? i : 2 * i - 1) : 2 * i + is_v);
          const uint32_t slot = ld % LY::KV_SLOTS, par = (ld / LY::KV_SLOTS) & 1u;
          if (ld >= (uint32_t)LY::KV_SLOTS) {
            const uint32_t u = SPLIT ? ld - LY::KV_SLOTS : (ld - LY::KV_SLOTS + 1) >> 1;
            ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->kv_release[u % LY::KV_SLOTS]),
                                                  (u / LY::KV_SLOTS) & 1u, abort_flag, p));
            if (!ok) break;
          }
          const uint32_t full = smem_u32(&bars->kv_full[slot]);
          const int keys = it.len - j * BN;  // boxes that hold a key of the sequence
          const int live = keys <= 0 ? 0 : min(boxes, (keys + p.box_keys - 1) / p.box_keys);
          if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)live * LY::CHUNKS * box_bytes);
          __syncwarp();
          if (issues && my_box < live)
            tma_load_4d(sKV + slot * LY::TILE_BYTES + box_off, tm, full, my_chunk * 64,
                        p.page_size > BN ? j % tiles_per_page * BN : 0, it.h, page);
          issued_mask |= 1u << slot;
          last_par = (last_par & ~(1u << slot)) | (par << slot);
          if (!is_v && i == 0) {  // Q behind the first K
            ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->q_empty), q_ph ^ 1, abort_flag, p));
            if (!ok) break;
            q_ph ^= 1;
            const uint32_t qf = smem_u32(&bars->q_full);
            const int tiles = SPLIT ? 1 : (it.nt > p.tpt ? 2 : 1);
            if (lane == 0)
              mbar_arrive_expect_tx(qf, (uint32_t)(tiles * REP * LY::CHUNKS * p.tpt * p.G) * 128u);
            __syncwarp();
            if (lane < tiles * REP * LY::CHUNKS) {
              const int c = lane % LY::CHUNKS, a = lane / LY::CHUNKS;  // a: copy (SPLIT) or tile (PAIR)
              const uint32_t off = SPLIT ? (uint32_t)a * (BM / REP) * 128u : (uint32_t)a * LY::TILE_BYTES;
              tma_load_3d(sQ + off + c * LY::CHUNK_BYTES, &tmQ, qf, c * 64, it.h * p.G,
                          it.tok0 + (SPLIT ? 0 : a * p.tpt));
            }
            q_issued = true;
          }
        }
        ld0 += 2 * it.n;
      }
      if (!ok && lane == 0) {
        // every issued copy must land before the block may exit
        for (int s = 0; s < LY::KV_SLOTS; ++s)
          if (issued_mask & (1u << s)) wait_drain(smem_u32(&bars->kv_full[s]), (last_par >> s) & 1u, p);
        if (q_issued) wait_drain(smem_u32(&bars->q_full), q_ph ^ 1, p);
      }
      __syncwarp();
    } else if (warp == WARP_MMA) {
      // ======================================================================= MMA issuer
      constexpr uint32_t ID_S = umma_idesc_f16(BF16 ? 1 : 0, 0, 0, BM, BN);
      constexpr uint32_t ID_O = umma_idesc_f16(BF16 ? 1 : 0, 0, 1, BM, D);
      const uint64_t dQ0 = umma_smem_desc(sQ, 16, 1024), dK = umma_smem_desc(sKV, 16, 1024);
      const uint64_t dV = umma_smem_desc(sKV, LY::CHUNK_BYTES, 1024);
      uint32_t q_ph = 0, p_ph[2] = {0, 0};
      bool ok = true;
      Item it = {};
      auto wait_all = [&](uint32_t bar, uint32_t par) -> bool {
        return __all_sync(0xffffffffu, wait_bar(bar, par, abort_flag, p));
      };
      auto kv_wait = [&](uint32_t ld, uint32_t& slot) -> bool {
        slot = ld % LY::KV_SLOTS;
        return wait_all(smem_u32(&bars->kv_full[slot]), (ld / LY::KV_SLOTS) & 1u);
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(smem_u32(bar));
        __syncwarp();
      };
      auto issue_s = [&](int q_tile, int g, uint32_t kslot) {
        const uint64_t dq = dQ0 + ((q_tile * LY::TILE_BYTES) >> 4), dk = dK + ((kslot * LY::TILE_BYTES) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * LY::CHUNK_BYTES + (ks & 3) * 32) >> 4;
            umma_ss(tmem + TMEM_S0 + g * 128, dq + off, dk + off, ID_S, ks > 0 ? 1u : 0u);
          }
        }
        __syncwarp();
      };
      auto issue_pv = [&](int g, uint32_t vslot, bool acc) {
        const uint64_t dv = dV + ((vslot * LY::TILE_BYTES) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks)
            umma_ts(tmem + TMEM_O0 + g * 128, tmem + TMEM_S0 + g * 128 + ks * 8, dv + ((ks * 16 * 128) >> 4), ID_O,
                    (acc || ks > 0) ? 1u : 0u);
        }
        __syncwarp();
      };
      // What lies behind the sequence's last key in its last tile may be anything, NaN included,
      // and P's zeros there do not silence it: those rows of V become zeros before the product.
      auto clear_tail = [&](int j, uint32_t vslot) {
        const long long keys = it.len - (long long)j * BN;
        if (keys >= BN) return;
        const int from = keys < 0 ? 0 : (int)keys;
        const uint32_t base = sKV + vslot * LY::TILE_BYTES;
        for (int x = from * 8 + lane; x < BN * 8; x += 32) {  // 16-byte pieces of 128-byte rows
#pragma unroll
          for (int c = 0; c < LY::CHUNKS; ++c) st_shared_v4(base + c * LY::CHUNK_BYTES + x * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      uint32_t ld = 0;  // SPLIT: next load; PAIR: loads of the pieces before (K_i is ld + 2i)
      while (ok) {
        const Item* src = item_next();
        if (!(ok = src != nullptr)) break;
        it = *src;
        item_done();
        if (it.n == 0) break;
        uint32_t sK, sV;
        ok = wait_all(smem_u32(&bars->q_full), q_ph);
        if (!ok) break;
        q_ph ^= 1;
        if constexpr (SPLIT) {
          auto next_s = [&](int i) -> bool {  // S of tile i into buffer i & 1
            if (!kv_wait(ld, sK)) return false;
            tc_fence_after();
            issue_s(0, i & 1, sK);
            commit(&bars->s_full[i & 1]);
            commit(&bars->kv_release[ld % LY::KV_SLOTS]);
            if (i == it.n - 1) commit(&bars->q_empty);
            ++ld;
            return true;
          };
          ok = next_s(0) && (it.n < 2 || next_s(1));
          for (int i = 0; i < it.n && ok; ++i) {
            const int g = i & 1;
            ok = kv_wait(ld, sV);
            if (!ok) break;
            clear_tail(it.j0 + i, sV);
            ok = wait_all(smem_u32(&bars->p_full[g]), p_ph[g]);
            if (!ok) break;
            p_ph[g] ^= 1;
            tc_fence_after();
            issue_pv(g, sV, i >= 2);
            commit(&bars->kv_release[ld % LY::KV_SLOTS]);
            ++ld;
            // S(i+2) follows PV(i) in issue order, so its commit also says that O~_g is up to date
            if (i + 2 < it.n) ok = next_s(i + 2);
            else commit(&bars->o_done[g]);
          }
        } else {
          const bool has1 = it.nt > p.tpt;
          const int n0 = it.n0;
          ok = kv_wait(ld, sK);
          if (!ok) break;
          tc_fence_after();
          const uint32_t m = ld >> 1;
          issue_s(0, 0, sK);
          commit(&bars->s_full[0]);
          if (has1) {
            issue_s(1, 1, sK);
            commit(&bars->s_full[1]);
          }
          commit(&bars->kv_release[m % LY::KV_SLOTS]);
          if (it.n == 1) commit(&bars->q_empty);
          for (int i = 0; i < it.n; ++i) {
            const bool has_next = i + 1 < it.n;
            uint32_t sKn = 0;
            bool have_kn = false;
            auto wait_kn = [&]() -> bool {
              if (!have_kn) {
                if (!kv_wait(ld + 2 * i + 2, sKn)) return false;
                have_kn = true;
                tc_fence_after();
              }
              return true;
            };
            ok = kv_wait(ld + 2 * i + 1, sV);
            if (!ok) break;
            clear_tail(it.j0 + i, sV);
            if (i < n0) {
              ok = wait_all(smem_u32(&bars->p_full[0]), p_ph[0]);
              if (!ok) break;
              p_ph[0] ^= 1;
              tc_fence_after();
              issue_pv(0, sV, i > 0);
              if (i + 1 < n0) {
                ok = wait_kn();
                if (!ok) break;
                issue_s(0, 0, sKn);
                commit(&bars->s_full[0]);
              } else {
                commit(&bars->o_done[0]);
              }
            }
            if (has1) {
              ok = wait_all(smem_u32(&bars->p_full[1]), p_ph[1]);
              if (!ok) break;
              p_ph[1] ^= 1;
              tc_fence_after();
              issue_pv(1, sV, i > 0);
              if (has_next) {
                ok = wait_kn();
                if (!ok) break;
                issue_s(1, 1, sKn);
                commit(&bars->s_full[1]);
              } else {
                commit(&bars->o_done[1]);
              }
            }
            if (has_next) {
              ok = wait_kn();  // K of the next tile is in hand before its unit is given back
              if (!ok) break;
              commit(&bars->kv_release[(m + i + 1) % LY::KV_SLOTS]);
            }  // the piece's last V is released with the next piece's first K
            if (i + 2 == it.n) commit(&bars->q_empty);
          }
          ld += 2 * it.n;
        }
      }
      commit(&bars->mma_drain);
      wait_drain(smem_u32(&bars->mma_drain), 0, p);
      __syncwarp();
    } else if (warp == WARP_WALK) {
      // ======================================================================= items
      if (lane == 0) {
        int* rec = p.records + blockIdx.x * 8;
        rec[0] = 0;  // no item begins here and ends elsewhere, as yet
        Walk<TPT_MUL> walk;
        walk.begin(p, range, bars);
        for (uint32_t i = 0;; ++i) {
          const uint32_t s = i % ITEM_SLOTS;
          if (i >= ITEM_SLOTS && !wait_bar(smem_u32(&bars->item_empty[s]), (i / ITEM_SLOTS - 1) & 1u, abort_flag, p)) break;
          Item it;
          int last;
          const bool more = walk.next(p, range, it, last);
          if (!more) it.n = 0;
          bars->items[s] = it;
          mbar_arrive(smem_u32(&bars->item_full[s]));
          if (!more) break;
          if (it.j0 == 0 && it.n != it.ntot) {
            rec[1] = it.slot;
            rec[2] = last;
            rec[3] = it.h;
            rec[4] = it.tok0;
            rec[5] = it.nt;
            rec[0] = 1;
          }
        }
      }
      __syncwarp();
    }
    tc_fence_before();
    named_bar_sync(1, NUM_THREADS);
    if (warp == WARP_MMA) {
      tc_fence_after();
      tmem_dealloc(tmem, TMEM_COLS);
    }
  } else {
    regs_inc<REGS_SOFTMAX>();
    // ======================================================================= softmax
    const int g = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
    const int copy = r / (BM / REP), row = r % (BM / REP);  // REP = 1: copy 0, row r
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + TMEM_S0 + g * 128, tO = tmem + lane_off + TMEM_O0 + g * 128;
    const float c = p.c;
    uint32_t s_ph = 0, o_ph = 0, e_ph = 0;
    bool ok = true;
    // both warpgroups (8 warps)
    auto epi_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->epi));
      const bool w = wait_bar(smem_u32(&bars->epi), e_ph, abort_flag, p);
      e_ph ^= 1;
      return __all_sync(0xffffffffu, w);
    };
    while (ok) {
      const Item* item = item_next();
      if (!(ok = item != nullptr) || item->n == 0) break;
      const int tok = row / p.G + (SPLIT ? 0 : g * p.tpt);  // token of this row in the item
      const bool valid = row < p.tpt * p.G && tok < item->nt;
      if (!SPLIT && g == 1 && item->nt <= p.tpt) {
        item_done();
        continue;
      }
      // keys [0, lim) are visible; counted from the piece's first tile
      const int lim = (!valid ? 0 : p.causal ? max(0, min(item->vis0 + tok, item->len)) : item->len) - item->j0 * BN;
      const int n_my = !SPLIT && g == 0 ? item->n0 : item->n;
      float m_run = -INFINITY, l_run = 0.f;
      for (int i = SPLIT ? g : 0; i < n_my; i += SPLIT ? 2 : 1) {
        ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->s_full[g]), s_ph, abort_flag, p));
        if (!ok) break;
        s_ph ^= 1;
        tc_fence_after();
        uint32_t sr[CW / 32][32];
#pragma unroll
        for (int q = 0; q < CW / 32; ++q) tmem_ld32(tS + copy * CW + q * 32, sr[q]);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < CW / 32; ++q) reg_fence(sr[q]);
        auto sv = [&](int k) { return __uint_as_float(sr[k >> 5][k & 31]); };
        const int vis = lim - i * BN - copy * CW;
        // rows that hold no query do not decide which path the warp takes
        const bool full = __all_sync(0xffffffffu, !valid || vis >= CW);
        float mt;
        {
          constexpr int NT = (CW + 2) / 3;
          float t[NT];
          if (full) {
#pragma unroll
            for (int x = 0; x < NT; ++x)
              t[x] = max3(sv(3 * x), 3 * x + 1 < CW ? sv(3 * x + 1) : -INFINITY, 3 * x + 2 < CW ? sv(3 * x + 2) : -INFINITY);
          } else {
            auto mv = [&](int e) { return e < vis ? sv(e) : -INFINITY; };
#pragma unroll
            for (int x = 0; x < NT; ++x)
              t[x] = max3(mv(3 * x), 3 * x + 1 < CW ? mv(3 * x + 1) : -INFINITY, 3 * x + 2 < CW ? mv(3 * x + 2) : -INFINITY);
          }
          mt = tree_max<NT>(t);
        }
        const float m_tile = (mt == -INFINITY || !valid) ? -INFINITY : mt * c;
        float m_new = m_run, alpha = 1.f;
        bool rescale = false;
        if (i < (SPLIT ? 2 : 1)) {
          m_new = m_tile;
        } else if (m_tile > m_run + RESCALE_THRESHOLD) {
          m_new = m_tile;
          alpha = ex2_approx(m_run - m_new);
          rescale = true;
        }
        const float nb = (m_new == -INFINITY) ? 0.f : -m_new;
        const uint64_t c2 = f2(c, c), nb2 = f2(nb, nb);
        uint64_t acc[4] = {0, 0, 0, 0};
        uint32_t pk[CW / 2];
        if (full) {
#pragma unroll
          for (int k = 0; k < CW / 2; ++k) {
            float t0, t1;
            f2_split(f2_fma(f2(sv(2 * k), sv(2 * k + 1)), c2, nb2), t0, t1);
            const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
            acc[k & 3] = f2_add(acc[k & 3], f2(p0, p1));
            pk[k] = pack2<BF16>(p0, p1);
          }
        } else {
#pragma unroll
          for (int k = 0; k < CW / 2; ++k) {
            float t0, t1;
            f2_split(f2_fma(f2(sv(2 * k), sv(2 * k + 1)), c2, nb2), t0, t1);
            const float p0 = 2 * k < vis ? ex2_approx(t0) : 0.f;
            const float p1 = 2 * k + 1 < vis ? ex2_approx(t1) : 0.f;
            acc[k & 3] = f2_add(acc[k & 3], f2(p0, p1));
            pk[k] = pack2<BF16>(p0, p1);
          }
        }
        float a0, a1;
        f2_split(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
        if (__any_sync(0xffffffffu, rescale)) {
          const uint64_t al2 = f2(alpha, alpha);
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tO + q * 32, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x0, x1;
              f2_split(f2_mul(f2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), al2), x0, x1);
              o[2 * k] = __float_as_uint(x0);
              o[2 * k + 1] = __float_as_uint(x1);
            }
            tmem_st32(tO + q * 32, o);
          }
        }
        l_run = l_run * alpha + a0 + a1;
        m_run = m_new;
        // P over the first 64 columns of the scores: this copy's keys, zeros for the other copies'
        if constexpr (REP == 1) {
          tmem_st32(tS, reinterpret_cast<const uint32_t(&)[32]>(pk[0]));
          tmem_st32(tS + 32, reinterpret_cast<const uint32_t(&)[32]>(pk[32]));
        } else {
          uint32_t zero[16] = {};
          if constexpr (REP == 2) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              tmem_st16(tS + copy * 32 + hh * 16, pk + hh * 16);
              tmem_st16(tS + (copy ^ 1) * 32 + hh * 16, zero);
            }
          } else {
            tmem_st16(tS + copy * 16, pk);
#pragma unroll
            for (int x = 1; x < 4; ++x) tmem_st16(tS + ((copy + x) & 3) * 16, zero);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[g]));
      }
      if (!ok) break;
      // ------------------------------------------------------------------ epilogue
      const bool worked = !SPLIT || item->n > g;
      if (worked) {
        ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->o_done[g]), o_ph, abort_flag, p));
        if (!ok) break;
        o_ph ^= 1;
        tc_fence_after();
      }
      const bool partial = item->n != item->ntot;
      float* part = p.parts + (size_t)(blockIdx.x * 2 + item->slot) * part_floats(D, ROWS);
      if constexpr (!SPLIT) {
        const int prow = g * BM + row;
        const long long t = item->tok0 + tok;
        const int head = item->h * p.G + row % p.G;
        if (partial) {
          if (valid) *reinterpret_cast<float2*>(part + ROWS * D + 2 * prow) = make_float2(m_run, l_run);
        } else if (valid && p.L) {
          p.L[t * (p.Hkv * p.G) + head] = l_run > 0.f ? (m_run + log2f(l_run)) * 0.69314718055994531f : -INFINITY;
        }
        const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
        uint16_t* orow = p.o.ptr + t * p.o.ts + (long long)head * p.o.hs;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(tO + q * 32, o);
          tmem_wait_ld();
          reg_fence(o);
          if (valid && partial) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              reinterpret_cast<uint4*>(part + (size_t)prow * D + q * 32)[k] =
                  make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          } else if (valid) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(o[8 * k + e]) * inv;
              reinterpret_cast<uint4*>(orow + q * 32)[k] = pack8<BF16>(x);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
      } else {
        // The row's 2 REP states (two warpgroups, REP copies) become one: their (m, l) meet in
        // the stage, then the second warpgroup's scaled O~, then the sums of both.
        st_shared_u32(sStage + (uint32_t)((g * BM + r) * 8), __float_as_uint(m_run));
        st_shared_u32(sStage + (uint32_t)((g * BM + r) * 8 + 4), __float_as_uint(l_run));
        if (!(ok = epi_sync())) break;
        const float2* states = reinterpret_cast<const float2*>(smem + LY::OFF_STAGE);
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int x = 0; x < 2 * REP; ++x) m = fmaxf(m, states[x * (BM / REP) + row].x);
        auto scale_of = [&](float mx) { return mx == -INFINITY ? 0.f : ex2_approx(mx - m); };
#pragma unroll
        for (int x = 0; x < 2 * REP; ++x) {
          const float2 st = states[x * (BM / REP) + row];
          l += st.y * scale_of(st.x);
        }
        // a whole item's O is divided by l here already; a partial state stays as it is
        const float f = scale_of(m_run) * (partial ? 1.f : l > 0.f ? 1.f / l : 0.f);
        if (!(ok = epi_sync())) break;
        // 16-byte piece x of row r stands at place x ^ (r & 7)
        auto stage_at = [&](int rr, int x) { return sStage + (uint32_t)(rr * D * 4 + ((x ^ (rr & 7)) << 4)); };
        auto put = [&](bool add) {
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tO + q * 32, o);
            tmem_wait_ld();
            reg_fence(o);
            if (valid) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                float x[4] = {};
                if (add) ld_shared_v4(stage_at(r, q * 8 + k), x);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = fmaf(__uint_as_float(o[4 * k + e]), f, x[e]);
                st_shared_v4(stage_at(r, q * 8 + k), __float_as_uint(x[0]), __float_as_uint(x[1]),
                             __float_as_uint(x[2]), __float_as_uint(x[3]));
              }
            }
            __syncwarp();
          }
        };
        if (g == 1 && worked) put(false);
        if (!(ok = epi_sync())) break;
        if (g == 0) put(item->n > 1);
        tc_fence_before();
        const long long t = item->tok0 + tok;
        const int head = item->h * p.G + row % p.G;
        if (g == 0 && copy == 0 && valid) {
          if (partial) *reinterpret_cast<float2*>(part + ROWS * D + 2 * row) = make_float2(m, l);
          else if (p.L) p.L[t * (p.Hkv * p.G) + head] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
        if (!(ok = epi_sync())) break;
        // sums of the copies: thread = 8 columns of a row
        const int rows = min(item->nt, p.tpt) * p.G;
        for (int x = threadIdx.x; x < rows * (D / 8); x += 256) {
          const int rr = x / (D / 8), c8 = x % (D / 8);
          float sum[8] = {};
#pragma unroll
          for (int a = 0; a < REP; ++a) {
            float y[4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              ld_shared_v4(stage_at(a * (BM / REP) + rr, 2 * c8 + hh), y);
#pragma unroll
              for (int e = 0; e < 4; ++e) sum[4 * hh + e] += y[e];
            }
          }
          if (partial) {
            float4* dst = reinterpret_cast<float4*>(part + (size_t)rr * D + 8 * c8);
            dst[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
            dst[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
          } else {
            const long long tt = item->tok0 + rr / p.G;
            uint16_t* dst = p.o.ptr + tt * p.o.ts + (long long)(item->h * p.G + rr % p.G) * p.o.hs + 8 * c8;
            *reinterpret_cast<uint4*>(dst) = pack8<BF16>(sum);
          }
        }
        if (!(ok = epi_sync())) break;
      }
      item_done();
    }
    tc_fence_before();
    named_bar_sync(1, NUM_THREADS);
  }
}

// Joins the partial states of the items that lie in several blocks' ranges: blocks (c, y) take
// the item that begins in block c's range, one warp per row.
template <int D, bool BF16, int ROWS>
__global__ void __launch_bounds__(COMBINE_THREADS) fa_paged_combine_kernel(const __grid_constant__ Params p) {
  constexpr int E = D / 32;  // columns per lane
  wait_previous_grid();
  const int* rec = p.records + blockIdx.x * 8;
  if (rec[0] == 0) return;
  const int c0 = blockIdx.x, slot0 = rec[1], c1 = rec[2], h = rec[3], tok0 = rec[4], nt = rec[5];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hq = p.Hkv * p.G, n = c1 - c0 + 1;
  auto part = [&](int x) {  // piece x of the item
    return p.parts + (size_t)((c0 + x) * 2 + (x == 0 ? slot0 : 0)) * part_floats(D, ROWS);
  };
  for (int pr = blockIdx.y * (COMBINE_THREADS / 32) + warp; pr < ROWS; pr += gridDim.y * (COMBINE_THREADS / 32)) {
    const int row = pr % BM, tok = row / p.G + pr / BM * p.tpt;
    if (row >= p.tpt * p.G || tok >= nt) continue;
    float m = -INFINITY, l = 0.f;
    for (int x = lane; x < n; x += 32) m = fmaxf(m, part(x)[ROWS * D + 2 * pr]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float acc[E] = {};
    for (int x0 = 0; x0 < n; x0 += 32) {
      float w = 0.f;
      if (x0 + lane < n) {
        const float2 st = *reinterpret_cast<const float2*>(part(x0 + lane) + ROWS * D + 2 * pr);
        if (st.x != -INFINITY) w = ex2_approx(st.x - m);
        l += st.y * w;
      }
      const int k = min(32, n - x0);
#pragma unroll 4
      for (int y = 0; y < k; ++y) {
        const float wy = __shfl_sync(0xffffffffu, w, y);
        const float* src = part(x0 + y) + (size_t)pr * D + lane * E;
        float v[E];
        if constexpr (E == 4) {
          const float4 q = *reinterpret_cast<const float4*>(src);
          v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
          const float2 q = *reinterpret_cast<const float2*>(src);
          v[0] = q.x, v[1] = q.y;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = wy != 0.f ? fmaf(v[e], wy, acc[e]) : acc[e];
      }
    }
    l = row_sum<32>(l);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const long long t = tok0 + tok;
    const int head = h * p.G + row % p.G;
    uint16_t* dst = p.o.ptr + t * p.o.ts + (long long)head * p.o.hs + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack2<BF16>(acc[e] * inv, acc[e + 1] * inv);
    if (p.L && lane == 0) p.L[t * Hq + head] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace paged
}  // namespace fa
