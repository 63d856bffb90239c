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
// Work. An item is (sequence, key head, block of tokens); its keys are cut into tiles of 128. It
// counts as one unit per tile and ITEM_UNITS before them for what an item costs by itself. The
// lengths are device data, so every block adds up the units of all sequences by itself (a closed
// form per sequence), and block c of Ge takes the units [c W / Ge, (c+1) W / Ge) of the W in order.
// An item whose tiles lie in several blocks' ranges leaves partial states (m, l, O~) in the
// workspace; fa_paged_combine_kernel joins them, in the order of the blocks. Nothing in the main
// kernel waits on another block. Where the table is so narrow that no item has more than
// WHOLE_TILES tiles, items stay whole and the second kernel falls away: an item of 4 tiles by one
// block takes 1 us more than by two, less than the second kernel costs; with whole items of up to 8
// tiles one token over 1000 keys took 2.5 us more, fresh prompts of 1000 tokens 2 less.
// Small batches go without units at all ("direct"): one sequence of single tokens, whose key heads
// share the SMs evenly, or whole items that fit the SMs at once. Block c then is part c % direct of
// (sequence, key head) c / direct, a range of its keys or one of its blocks of tokens, and reads the
// lengths of its own sequence only: 1 us less before the first load.
//
// Two forms of the kernel, of 12 warps (8, 11: loads, 9: MMA issuer, 10: walks the block's range and
// hands the others their items through a ring in shared memory, a few ahead, so that nobody waits
// for the lengths of the next sequence; 0-7: two softmax warpgroups, thread = row = TMEM lane):
//   PAIR   an item is two tiles of 128 rows, one per warpgroup, over the same keys: chunks. d = 128 is
//          bound by the tensor cores and the chain S - softmax - P V, d = 64 by that chain, with no pipe
//          full (exponentials 34 % of theirs, tensor cores 31 %, instruction issue 39 %). 2048 tokens
//          at 30720, Hq 16, Hkv 2, d 128: 326 to 330 us replayed in a graph, 1.62 PFLOP/s, and 341 to
//          354 us called one by one; 4 x 1000 over 4097 keys, 12 heads, d 64: 76 us, 0.66 PFLOP/s.
//   SPLIT  an item is one tile; the warpgroups take the even and the odd key tiles, each with its
//          own (m, l, O~). Its rows stand REP times in the tile (REP = 4 for up to 32 rows): copy
//          a covers keys [a 128/REP, (a+1) 128/REP) of each key tile only, with its own (m, l, O~)
//          and zeros in P elsewhere. So each warp reads 128/REP scores of each row instead of one
//          warp reading 128; nothing is exchanged before the item's end. Single tokens and
//          drafts: bound by HBM; the tensor cores run mostly empty and still hide behind the
//          loads (1024 cycles of products per 64 KB of keys and values, which take 2900 at this
//          SM's share of the bandwidth). 64 sequences of 201 to 8020 keys, 8 key heads, d 128, pages
//          of 16: 163 to 165 us, 6.4 TB/s; one sequence of 1001 keys: 9.5 us with the join, latency.
#pragma once

#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "fa_rope.cuh"

namespace fa {
namespace paged {

constexpr int BM = 128, BN = 128;
constexpr int NUM_WARPS = 12, NUM_THREADS = NUM_WARPS * 32;
constexpr int WARP_LOAD = 8, WARP_MMA = 9, WARP_WALK = 10, WARP_LOAD2 = 11;
constexpr int ITEM_SLOTS = 4;
constexpr int ITEM_READERS = 11;  // warps that read an item: two loading, MMA, 8 softmax
// Waits on the ring of items last as long as an item, up to thousands of key tiles, while the limit is
// meant for a step of the pipeline: they have this many times it. (Where the pipeline stands still, one
// of its own waits runs out first and stops these as well.)
constexpr uint32_t ITEM_WAITS = 1024;
// 2*128*200 + 128*104 = 64512 = 384*168 registers, the launch's budget
constexpr uint32_t REGS_SOFTMAX = 200, REGS_OTHER = 104;
constexpr uint32_t TMEM_COLS = 512, TMEM_S0 = 0, TMEM_O0 = 256;  // S0 | S1 | O0 | O1
constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units, as in the dense kernel
constexpr int SMEM_LIMIT = 232448;
constexpr int MAX_SLOTS = 8;
constexpr int COMBINE_THREADS = 256;
constexpr int WHOLE_TILES = FA_PAGED_WHOLE_KEYS / BN;
// units of a block at least: with 1, more pieces of an item to join than the shorter pieces gain, with 5
// the pieces are long (at least 1, 2, 3, 5 units: 100 tokens of 8 heads over 4000 keys of one, d 128,
// 22.5, 20.0, 20.4, 22.3 us; three sequences of 1001 keys of 8 heads, d 128, 12.0, 11.6, 12.4, 13.9 us)
constexpr int MIN_UNITS = 3;
// key tiles of a part at least, one for each warpgroup (one sequence of 1001 keys: 9.5 us, with 1 tile
// 9.7, with 3 10.7)
constexpr int DIRECT_TILES = 2;

struct Params {
  HeadsDev o;
  float* L;
  int num_pages, page_size, box_keys;  // box_keys: keys per TMA box, min(page_size, 128)
  int Hkv, G, tpt;                     // tpt: tokens per tile, (128 / REP) / G
  uint32_t by_g;                       // ceil(2^16 / G): row / G = row * by_g >> 16, exact for row, G <= 128
  const int *cu, *lens, *table;
  int table_stride, B, T, causal;
  int cap;    // keys that a row of the table covers
  int whole;  // no item is split: a block takes the items that begin in its range
  int direct; // that many blocks to a (sequence, key head), without units (0: by units)
  float c;  // scale * log2(e)
  unsigned long long wait_limit_ns;
  int* status;
  int* records;  // [block][8]: the item that begins in a block's range and ends in another's (7 in use)
  float* parts;  // [block][2][rows]: D floats of O~ per row, then [rows][2] of (m, l)
  long long parts_len;  // floats there (checked by debug builds)
};

// Debug builds (FA_DEBUG) check the places of tile copies, partial states and output rows; one
// outside records FA_ERR_BOUNDS. Stores, and the join of an item whose pieces it concerns, are then
// skipped; a tile copy is only recorded (TMA reads zeros outside, and its barrier expects the bytes).
// Release builds compile it out.
__device__ __forceinline__ bool in_bounds(const Params& p, bool ok) {
#ifdef FA_DEBUG
  if (!ok) atomicCAS(p.status, 0, FA_ERR_BOUNDS);
  return ok;
#else
  (void)p, (void)ok;
  return true;
#endif
}

__device__ __forceinline__ int token_of_row(const Params& p, int row) { return (int)((uint32_t)row * p.by_g >> 16); }
__host__ __device__ constexpr int part_floats(int d, int rows) { return rows * (d + 2); }

// One block's part of one item.
struct Item {
  int b, h, tok0, nt;   // sequence, key head, first row of q, tokens
  int len, vis0;        // cached tokens; keys that the item's first token sees (causal)
  int j0, n, ntot;      // key tiles [j0, j0 + n) of ntot; n = 0: no more items
  int n0;               // PAIR: of the n, those that reach the first tile's rows (at least 1)
  int slot;             // place of its partial state: 0 = first piece of the block's range
};

struct Seq {
  int t0, n, len, nq;  // first row of q, new tokens, tokens in the cache, blocks of tokens
};
// Where a block's range begins: `rem` units into sequence b.
struct Start {
  long long rem;
  int b, h, q, off;  // off: units into the item
  Seq s;
};

struct Barriers {
  uint64_t q_full, q_empty;
  uint64_t kv_full[MAX_SLOTS], kv_release[MAX_SLOTS];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t mma_drain, epi;
  uint64_t item_full[ITEM_SLOTS], item_empty[ITEM_SLOTS];
  Item items[ITEM_SLOTS];
  long long warp_units[NUM_WARPS];
  Start start;
  uint32_t tmem_base;
  int abort_flag;
};

template <int D, bool SPLIT>
struct Layout {
  static constexpr int TILE_BYTES = BM * D * 2;
  static constexpr int CHUNK_BYTES = BM * 128, CHUNKS = D / 64;
  static constexpr int Q_TILES = SPLIT ? 1 : 2;
  // SPLIT: fp32 rows of O~. PAIR: 4 KB per softmax warp, 32 rows of 128 bytes on their way out.
  static constexpr int STAGE_BYTES = SPLIT ? 65536 : 32768;
  static constexpr int STAGE_ROWS = STAGE_BYTES / (D * 4);
  static constexpr int STATE_BYTES = SPLIT ? 2 * BM * 8 : 0;  // (m, l) of both warpgroups' rows
  static constexpr int HEAD_BYTES = 1024;                     // barriers and items
  static constexpr int FIT =
      (SMEM_LIMIT - Q_TILES * TILE_BYTES - STAGE_BYTES - STATE_BYTES - HEAD_BYTES) / TILE_BYTES;
  static constexpr int KV_SLOTS = FIT > MAX_SLOTS ? MAX_SLOTS : FIT;
  static constexpr int OFF_Q = 0, OFF_KV = Q_TILES * TILE_BYTES;
  static constexpr int OFF_STAGE = OFF_KV + KV_SLOTS * TILE_BYTES;
  static constexpr int OFF_STATE = OFF_STAGE + STAGE_BYTES;
  static constexpr int OFF_BAR = OFF_STATE + STATE_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + HEAD_BYTES;
  static_assert(sizeof(Barriers) <= 1024 && KV_SLOTS >= 4 && SMEM_BYTES <= SMEM_LIMIT, "shared memory budget");
};

// ----------------------------------------------------------------------------- waits
// Bounded: a wait past the limit records FA_ERR_TIMEOUT and stops every role of the block.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, const Params& p,
                                          uint32_t limits) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > p.wait_limit_ns * limits) {
      atomicCAS(p.status, 0, FA_ERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, const Params& p,
                                         uint32_t limits = 1) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, abort_flag, p, limits);
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
// Sequence b as the kernels see it: a range of rows outside [0, T] counts as empty, a length
// past the table's width is cut to it; `report` records either.
__device__ __forceinline__ Seq load_seq(const Params& p, int b, int tpi, bool report) {
  Seq s;
  s.t0 = p.cu[b];
  const int end = p.cu[b + 1], len = p.lens[b];
  const bool rows_ok = s.t0 >= 0 && end >= s.t0 && end <= p.T;
  s.n = rows_ok ? end - s.t0 : 0;
  s.len = max(0, min(len, p.cap));
  s.nq = s.n <= tpi ? (s.n > 0) : (s.n - 1) / tpi + 1;
  if (report && (!rows_ok || (s.n && len > p.cap))) atomicCAS(p.status, 0, FA_ERR_RANGE);
  return s;
}

// a / b for b > 0; nearly always 32 bits
__device__ __forceinline__ long long divide(long long a, int b) {
  return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// key tiles of a block of tokens that sees `vis` keys (at least one, so that its rows are written)
__device__ __forceinline__ int tiles_for(int vis) { return vis <= 0 ? 1 : (int)((uint32_t)(vis + BN - 1) / BN); }
// of block q
__device__ __forceinline__ int tiles_of(const Params& p, const Seq& s, int q, int tpi) {
  const uint32_t end = min((uint32_t)(q + 1) * (uint32_t)tpi, (uint32_t)s.n);
  return tiles_for(p.causal ? s.len - s.n + (int)end : s.len);
}

// Key tiles of the first q blocks. With a causal mask block i sees x_i = ctx + (i + 1) tpi keys
// (the last one all of them): the first k0 at most 128, one tile, and the others ceil(x_i / 128)
// = (x_i + r_i) / 128 tiles with r_i = -x_i mod 128. The r_i of 128 / g blocks in a row, g the
// largest power of two in tpi (up to 128), are rho, rho + g, rho + 2 g, ... in some order.
__device__ __forceinline__ long long tiles_before(const Params& p, const Seq& s, int q, int tpi) {
  if (q == 0) return 0;
  if (!p.causal) return (long long)q * tiles_for(s.len);
  if (q == 1) return tiles_of(p, s, 0, tpi);
  const int full = q < s.nq ? q : s.nq - 1;
  const long long ctx = (long long)s.len - s.n;
  long long k0 = ctx >= BN ? 0 : divide(BN - ctx, tpi);
  if (k0 > full) k0 = full;
  long long sum = k0;
  const long long n = full - k0, x0 = ctx + (k0 + 1) * tpi;
  if (n > 0) {
    const int g = min(tpi & -tpi, BN), lp = __ffs(BN / g) - 1, period = 1 << lp;
    long long r = (n >> lp) * ((long long)period * ((int)(-x0) & (g - 1)) + (long long)g * period * (period - 1) / 2);
#pragma unroll 1
    for (int i = (int)(n >> lp << lp); i < n; ++i) r += (int)(-(x0 + (long long)i * tpi)) & (BN - 1);
    sum += (n * x0 + tpi * (n * (n - 1) / 2) + r) / BN;
  }
  return sum + (q > full ? tiles_for(s.len) : 0);
}

struct Range {
  long long W, u0, u1;
  int Ge;  // blocks that take part
};
__device__ __forceinline__ long long bound_of(int c, const Range& r) { return divide(c * r.W, r.Ge); }
__device__ __forceinline__ int owner_of(long long u, const Range& r) {
  int c = (int)(u * r.Ge / r.W);
  while (c + 1 < r.Ge && bound_of(c + 1, r) <= u) ++c;
  return c;
}

// The item of block of tokens q of a sequence, key tiles [j0, j1).
template <int TPT_MUL>
__device__ __forceinline__ Item make_item(const Params& p, const Seq& s, int b, int h, int q, int ntot, int j0, int j1,
                                          int slot) {
  const int tpi = p.tpt * TPT_MUL;
  Item it;
  it.b = b;
  it.h = h;
  it.tok0 = s.t0 + q * tpi;
  it.nt = min(tpi, s.n - q * tpi);
  it.len = s.len;
  it.vis0 = s.len - s.n + q * tpi + 1;
  it.ntot = ntot;
  it.j0 = j0;
  it.n = j1 - j0;
  it.slot = slot;
  it.n0 = it.n;
  if (TPT_MUL == 2 && p.causal) {
    const int t = tiles_for(it.vis0 + min(p.tpt, it.nt) - 1) - j0;
    it.n0 = t < 1 ? 1 : min(t, it.n);
  }
  return it;
}

// Walks a block's range.
template <int TPT_MUL, int ITEM_UNITS>
struct Walk {
  Seq s;
  int b, h, q;
  long long u, off;  // next unit, and its place in its item
  bool first;
  __device__ __forceinline__ void begin(const Range& r, const Start& st) {
    s = st.s;
    b = st.b;
    h = st.h;
    q = st.q;
    off = st.off;
    u = r.u0;
    first = true;
  }
  // `ustart`: the item's first unit
  __device__ __forceinline__ bool next(const Params& p, const Range& r, Item& it, long long& ustart) {
    const int tpi = p.tpt * TPT_MUL;
    while (u < r.u1) {
      if (q == s.nq) {
        q = 0;
        if (++h == p.Hkv) {
          h = 0;
          do {
            if (++b >= p.B) return false;
            s = load_seq(p, b, tpi, false);
          } while (s.n == 0);
        }
      }
      const int ntot = tiles_of(p, s, q, tpi);
      const long long whole = ntot + ITEM_UNITS;
      const long long end = p.whole || off + (r.u1 - u) > whole ? whole : off + (r.u1 - u);
      const int j0 = off > ITEM_UNITS ? (int)(off - ITEM_UNITS) : 0;
      const int j1 = end > ITEM_UNITS ? (int)(end - ITEM_UNITS) : 0;
      ustart = u - off;
      u += end - off;
      off = 0;
      const int qq = q++;
      if (j1 == j0) continue;            // none of the item's tiles: they are the next block's
      if (p.whole && ustart < r.u0) continue;  // the block before has taken it
      it = make_item<TPT_MUL>(p, s, b, h, qq, ntot, j0, j1, first ? 0 : 1);
      first = false;
      return true;
    }
    return false;
  }
};

// units of the sequences of one thread, [b0, b1)
template <int TPT_MUL, int ITEM_UNITS>
__device__ __forceinline__ long long units_of(const Params& p, int b0, int b1, Seq& last, bool report) {
  const int tpi = p.tpt * TPT_MUL;
  long long sum = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    last = load_seq(p, b, tpi, report);
    sum += p.Hkv * (tiles_before(p, last, last.nq, tpi) + (long long)ITEM_UNITS * last.nq);
  }
  return sum;
}

// The block's share of the units, and where it begins (bars->start). All threads call this, with
// the units of their own sequences; it ends with a barrier.
template <int TPT_MUL, int ITEM_UNITS, int MIN_UNITS>
__device__ __forceinline__ Range plan(const Params& p, Barriers* bars, int b0, int b1, long long mine, Seq s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tpi = p.tpt * TPT_MUL;
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
  r.Ge = r.W < (long long)gridDim.x * MIN_UNITS ? ((int)r.W + MIN_UNITS - 1) / MIN_UNITS : (int)gridDim.x;
  r.u0 = r.u1 = 0;
  if ((int)blockIdx.x < r.Ge) {
    r.u0 = bound_of(blockIdx.x, r);
    r.u1 = bound_of(blockIdx.x + 1, r);
  }
  // the thread whose sequences hold the first unit
  if (r.u0 < r.u1 && before <= r.u0 && r.u0 < before + mine) {
    int b = b0;
    if (b1 - b0 > 1) {
#pragma unroll 1
      for (;; ++b) {
        const long long x = units_of<TPT_MUL, ITEM_UNITS>(p, b, b + 1, s, false);
        if (r.u0 < before + x) break;
        before += x;
      }
    }
    Start& st = bars->start;
    st.s = s;
    st.b = b;
    st.rem = r.u0 - before;
    if (s.nq == 1) {
      const int item = ITEM_UNITS + tiles_of(p, s, 0, tpi);
      st.h = (int)divide(st.rem, item);
      st.q = 0;
      st.off = (int)(st.rem - (long long)st.h * item);
    }
  }
  __syncthreads();
  if (r.u0 < r.u1 && bars->start.s.nq > 1) {  // the same for the whole block
    if (warp == 0) {
      Start& st = bars->start;
      s = st.s;
      const long long head = tiles_before(p, s, s.nq, tpi) + (long long)ITEM_UNITS * s.nq;
      const int h = (int)(st.rem / head);
      const long long rem = st.rem - h * head;
      // the last block with at most `rem` units before it: 32 candidates at a time
      int lo = 0, n = s.nq;
#pragma unroll 1
      while (n > 1) {
        const int step = (n + 31) / 32, cand = lo + lane * step;
        const bool le = lane * step < n && tiles_before(p, s, cand, tpi) + (long long)ITEM_UNITS * cand <= rem;
        const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;  // candidate 0 always holds
        lo += k * step;
        n = min(step, n - k * step);
      }
      if (lane == 0) {
        st.h = h;
        st.q = lo;
        st.off = (int)(rem - tiles_before(p, s, lo, tpi) - (long long)ITEM_UNITS * lo);
      }
    }
    __syncthreads();
  }
  return r;
}

// ----------------------------------------------------------------------------- kernel
// DIRECT: batches that go without units may come (SPLIT: always; PAIR has an instantiation with and
// one without that code, whose mere presence slowed the long chunks' loop from 339 to 351 us).
template <int D, bool BF16, bool SPLIT, int REP, bool DIRECT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    fa_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  static_assert(SPLIT || REP == 1, "copies of rows belong to the SPLIT form");
  using LY = Layout<D, SPLIT>;
  // ITEM_UNITS: what an item costs by itself, in key tiles. Against it, us: REP 4, 2 units: 24 drafts, d 64,
  // 35.8, with 1 41.6, with 4 36.6 (64 ragged single tokens, d 128: 165.0, 163.7, 166.3). REP 2, 3 units: 64
  // sequences of 16 tokens, d 128, 57.3, with 2 57.4, with 4 56.8. REP 1, 4 units: 256 of 32 tokens, d 64,
  // 37.7, with 2 40.2, with 6 37.3. PAIR, 2 units: 8 chunks, d 64, 36.8, with 1 37.2, with 4 38.5 (a chunk of
  // 2048 tokens, d 128: 328, 331, 334; fresh prompts of 2000 tokens 76.0, 74.6, 78.5).
  constexpr int TPT_MUL = SPLIT ? 1 : 2, ITEM_UNITS = SPLIT ? (REP == 1 ? 4 : REP == 2 ? 3 : 2) : 2;
  constexpr int ROWS = SPLIT ? BM / REP : 2 * BM;  // rows of an item's partial state
  constexpr int CW = BN / REP;                     // keys of a tile that one row copy covers
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;  // 1024-byte aligned, as the 128-byte swizzle wants it
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, FA_ERR_ALIGN);
    return;
  }
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
  wait_previous_grid();  // no global memory is read or written before this
  Range range = {};
  tc_fence_before();
  if (DIRECT && p.direct) {
    __syncthreads();
  } else {
    const int per_thread = (p.B + NUM_THREADS - 1) / NUM_THREADS;
    const int b0 = min((int)threadIdx.x * per_thread, p.B), b1 = min(b0 + per_thread, p.B);
    Seq seq = {};
    const long long my_units = units_of<TPT_MUL, ITEM_UNITS>(p, b0, b1, seq, blockIdx.x == 0);
    range = plan<TPT_MUL, ITEM_UNITS, MIN_UNITS>(p, bars, b0, b1, my_units, seq);
  }
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // Items in order: the reader's place in the ring, and the item there (nullptr: the wait gave up).
  uint32_t n_item = 0;
  auto item_next = [&]() -> const Item* {
    const uint32_t s = n_item % ITEM_SLOTS;
    const bool w = wait_bar(smem_u32(&bars->item_full[s]), (n_item / ITEM_SLOTS) & 1u, abort_flag, p,
                            ITEM_WAITS);
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
    // once. SPLIT: K0 K1 V0 K2 V1 K3 ...; every load is released by itself. Loads are released in
    // order, and two loads in a row of one warp are at most 3 apart: when a warp waits for the release
    // of load i - KV_SLOTS, those up to i - 3 - KV_SLOTS are past, so that the slot's barrier stands
    // in the phase waited for or behind it, never two phases before (where the parity would lie).
    if (warp == WARP_LOAD || warp == WARP_LOAD2) {
      // ======================================================================= producers
      // All 32 lanes: a tile's boxes (pages, and 64-column halves) are issued side by side. A box
      // costs its warp about 100 cycles whatever its size, 1600 for a tile's keys in pages of 16
      // (d = 128), so two warps share the work. SPLIT: the block's key tiles in turn, so that an item's
      // first two tiles are asked for at once (8 x 32768 keys of 8 heads, d 64, pages of 16: 93 us
      // against 100 with a warp for K and one for V; pages of 8, d 128: 186 against 203). PAIR: K and
      // V, which are used apart (32 prompts of 500 tokens, pages of 16: 64 us against 69 in turn).
      const uint32_t me = warp == WARP_LOAD2;
      const int boxes = BN / p.box_keys;                    // page boxes of one 64-column chunk
      const int tiles_per_page = p.page_size > BN ? p.page_size / BN : 1;
      const int my_box = lane % boxes, my_chunk = lane / boxes;
      const bool issues = my_chunk < LY::CHUNKS;
      const uint32_t box_bytes = (uint32_t)p.box_keys * 128u;
      const uint32_t box_off = (uint32_t)my_chunk * LY::CHUNK_BYTES + (uint32_t)my_box * box_bytes;
      uint32_t ld0 = 0, n_q = 0, issued_mask = 0, last_par = 0;  // n_q: Q loads of the items so far
      bool ok = true;
      // An item's Q, by the first of the two warps for every item: it has then waited for every
      // release of the buffer, and a parity cannot stand for one two phases back.
      auto load_q = [&](const Item& it) -> bool {
        if (!__all_sync(0xffffffffu, wait_bar(smem_u32(&bars->q_empty), (n_q & 1u) ^ 1u, abort_flag, p))) return false;
        const uint32_t qf = smem_u32(&bars->q_full);
        const int tiles = SPLIT ? 1 : (it.nt > p.tpt ? 2 : 1);
        if (lane == 0) mbar_arrive_expect_tx(qf, (uint32_t)(tiles * REP * LY::CHUNKS * p.tpt * p.G) * 128u);
        __syncwarp();
        in_bounds(p, it.tok0 >= 0 && it.tok0 + it.nt <= p.T && (it.h + 1) * p.G <= p.o.H);
        if (lane < tiles * REP * LY::CHUNKS) {
          const int c = lane % LY::CHUNKS, a = lane / LY::CHUNKS;  // a: copy (SPLIT) or tile (PAIR)
          const uint32_t off = SPLIT ? (uint32_t)a * (BM / REP) * 128u : (uint32_t)a * LY::TILE_BYTES;
          tma_load_3d(sQ + off + c * LY::CHUNK_BYTES, &tmQ, qf, c * 64, it.h * p.G, it.tok0 + (SPLIT ? 0 : a * p.tpt));
        }
        ++n_q;
        return true;
      };
      // 32 entries of a sequence's table, one per lane; -1 where one holds no key of the sequence,
      // num_pages (which reads as zeros) for a bad one
      auto ask = [&](int b, int window) -> int {
        const int e = window * 32 + lane;
        return e < p.table_stride ? p.table[(size_t)b * p.table_stride + e] : -1;
      };
      auto check = [&](int page, int len, int window) -> int {
        if ((long long)(window * 32 + lane) * p.page_size >= len) return -1;
        if (page >= 0 && page < p.num_pages) return page;
        atomicCAS(p.status, 0, FA_ERR_RANGE);
        return p.num_pages;
      };
      auto window_of = [&](int j) { return (p.page_size > BN ? j / tiles_per_page : j * boxes) / 32; };
      // those of the block's first tile are asked for before its item has been handed over
      int early_b = -1, early_window = 0, early = 0;
      if (DIRECT && p.direct) {
        if (p.whole) early_b = (int)blockIdx.x / p.direct / p.Hkv;
      } else if (range.u0 < range.u1) {
        early_b = bars->start.b;
        early_window = window_of(max(bars->start.off - ITEM_UNITS, 0));
      }
      if (early_b >= 0) early = ask(early_b, early_window);
      while (ok) {
        const Item* src = item_next();
        if (!(ok = src != nullptr)) break;
        const Item it = *src;
        item_done();
        if (it.n == 0) break;
        // the next 32 entries are always on their way
        auto entries = [&](int w) { return check(ask(it.b, w), it.len, w); };
        int window = window_of(it.j0);
        int held = it.b == early_b && window == early_window ? check(early, it.len, window) : entries(window);
        int next = entries(window + 1);
        early_b = -1;
        const int first_i = SPLIT ? (int)(((ld0 >> 1) ^ me) & 1u) : 0;
        if (me == 0 && first_i != 0 && !(ok = load_q(it))) break;
        for (int i = first_i; i < it.n && ok; i += SPLIT ? 2 : 1) {
          const int j = it.j0 + i;
          const int e0 = p.page_size > BN ? j / tiles_per_page : j * boxes;  // the tile's first entry
          if (e0 / 32 != window) {  // 32 is a multiple of a tile's entries
            held = e0 / 32 == window + 1 ? next : entries(e0 / 32);
            window = e0 / 32;
            next = entries(window + 1);
          }
          const int page = __shfl_sync(0xffffffffu, held, (e0 + my_box) % 32);
          const int keys = it.len - j * BN;  // boxes that hold a key of the sequence
          const int live = keys <= 0 ? 0 : min(boxes, (keys + p.box_keys - 1) / p.box_keys);
#pragma unroll(SPLIT ? 2 : 1)
          for (int is_v = SPLIT ? 0 : (int)me; is_v < (SPLIT ? 2 : (int)me + 1); ++is_v) {
            const uint32_t ld =
                ld0 + (SPLIT ? (is_v ? 2 + i + min(i, it.n - 2) : i < 2 ? i : 2 * i - 1) : 2 * i + is_v);
            const uint32_t slot = ld % LY::KV_SLOTS, par = (ld / LY::KV_SLOTS) & 1u;
            if (ld >= (uint32_t)LY::KV_SLOTS) {
              const uint32_t u = SPLIT ? ld - LY::KV_SLOTS : (ld - LY::KV_SLOTS + 1) >> 1;
              ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->kv_release[u % LY::KV_SLOTS]),
                                                    (u / LY::KV_SLOTS) & 1u, abort_flag, p));
              if (!ok) break;
            }
            const uint32_t full = smem_u32(&bars->kv_full[slot]);
            if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)live * LY::CHUNKS * box_bytes);
            __syncwarp();
            in_bounds(p, !issues || my_box >= live || (it.h < p.Hkv && page >= 0 && page <= p.num_pages));
            if (issues && my_box < live)
              tma_load_4d(sKV + slot * LY::TILE_BYTES + box_off, is_v ? &tmV : &tmK, full, my_chunk * 64,
                          p.page_size > BN ? j % tiles_per_page * BN : 0, it.h, page);
            issued_mask |= 1u << slot;
            last_par = (last_par & ~(1u << slot)) | (par << slot);
            // Q behind the first K
            if (me == 0 && is_v == 0 && i == 0 && !(ok = load_q(it))) break;
          }
        }
        ld0 += 2 * it.n;
      }
      if (!ok && lane == 0) {
        // every issued copy must land before the block may exit
        for (int s = 0; s < LY::KV_SLOTS; ++s)
          if (issued_mask & (1u << s)) wait_drain(smem_u32(&bars->kv_full[s]), (last_par >> s) & 1u, p);
        if (n_q) wait_drain(smem_u32(&bars->q_full), (n_q - 1) & 1u, p);
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
        if (!p.whole) rec[0] = 0;  // no item begins here and ends elsewhere, as yet
        uint32_t i = 0;
        auto publish = [&](const Item& it) -> bool {
          const uint32_t s = i % ITEM_SLOTS;
          if (i >= ITEM_SLOTS && !wait_bar(smem_u32(&bars->item_empty[s]), (i / ITEM_SLOTS - 1) & 1u, abort_flag, p,
                                           ITEM_WAITS))
            return false;
          bars->items[s] = it;
          mbar_arrive(smem_u32(&bars->item_full[s]));
          ++i;
          return true;
        };
        auto record = [&](const Item& it, int last) {  // its last block
          rec[1] = it.slot;
          rec[2] = last;
          rec[3] = it.h;
          rec[4] = it.tok0;
          rec[5] = it.nt;
          rec[6] = p.causal ? it.vis0 : it.len;  // keys that its first token sees
          rec[0] = 1;
        };
        bool go = true;
        if (DIRECT && p.direct) {
          const int item = (int)blockIdx.x / p.direct, part = (int)blockIdx.x - item * p.direct;
          const int b = item / p.Hkv, h = item - b * p.Hkv, tpi = p.tpt * TPT_MUL;
          const Seq s = load_seq(p, b, tpi, part == 0 && h == 0);
          // more blocks of tokens than the host knew of (max_q was too small): whole, by the last part
          // (whole items) or the first
          for (int q = p.whole ? part : 0; q < s.nq && go; ++q) {
            const int ntot = tiles_of(p, s, q, tpi);
            const int np = p.whole || q > 0 ? 1 : min(p.direct, (ntot + DIRECT_TILES - 1) / DIRECT_TILES);
            const int k = p.whole ? 0 : part;
            if (k >= np) continue;
            const uint32_t n = (uint32_t)ntot, j0 = k * n / np, j1 = (k + 1) * n / np;
            const Item it = make_item<TPT_MUL>(p, s, b, h, q, ntot, (int)j0, (int)j1, 0);
            go = publish(it);
            if (go && k == 0 && np > 1) record(it, (int)blockIdx.x + np - 1);
            if (p.whole && part < p.direct - 1) break;
          }
        } else {
          Walk<TPT_MUL, ITEM_UNITS> walk;
          walk.begin(range, bars->start);
          Item it;
          long long ustart;
          while (go && walk.next(p, range, it, ustart)) {
            go = publish(it);
            if (go && it.j0 == 0 && it.n != it.ntot) record(it, owner_of(ustart + ITEM_UNITS + it.ntot - 1, range));
          }
        }
        Item end = {};
        if (go) publish(end);
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
    const int row_tok = token_of_row(p, row), row_head = row - row_tok * p.G;
    const bool row_used = row < p.tpt * p.G;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + TMEM_S0 + g * 128, tO = tmem + lane_off + TMEM_O0 + g * 128;
    const float c = fmaxf(p.c, 1e-30f);  // a scale of zero: every finite score still counts as zero
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
      const int tok = row_tok + (SPLIT ? 0 : g * p.tpt);  // token of this row in the item
      // may a row of the item be stored, as output or in the block's partial state?
      auto storable = [&](int token, int head) {
        return in_bounds(p, item->tok0 >= 0 && item->tok0 + token < p.T && item->h * p.G + head < p.o.H &&
                                (item->n == item->ntot ||
                                 (blockIdx.x * 2 + item->slot + 1ll) * part_floats(D, ROWS) <= p.parts_len));
      };
      const bool valid = row_used && tok < item->nt && storable(tok, row_head);
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
        // Scores of keys that a row does not see become -inf, 32 columns at a time where some row of
        // the warp needs it (rows that hold no query do not count). c > 0 keeps them at -inf, and
        // their weights at zero.
        if (!__all_sync(0xffffffffu, !valid || vis >= CW)) {
#pragma unroll
          for (int q = 0; q < CW / 32; ++q) {
            if (__all_sync(0xffffffffu, !valid || vis >= 32 * (q + 1))) continue;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * q + k >= vis) sr[q][k] = 0xff800000u;
          }
        }
        float mt;
        {
          constexpr int NT = (CW + 2) / 3;
          float t[NT];
#pragma unroll
          for (int x = 0; x < NT; ++x)
            t[x] = max3(sv(3 * x), 3 * x + 1 < CW ? sv(3 * x + 1) : -INFINITY, 3 * x + 2 < CW ? sv(3 * x + 2) : -INFINITY);
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
#pragma unroll
        for (int k = 0; k < CW / 2; ++k) {
          float t0, t1;
          f2_split(f2_fma(f2(sv(2 * k), sv(2 * k + 1)), c2, nb2), t0, t1);
          const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
          acc[k & 3] = f2_add(acc[k & 3], f2(p0, p1));
          pk[k] = pack2<BF16>(p0, p1);
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
      const bool worked = !SPLIT || item->n > g, partial = item->n != item->ntot;
      // A row that sees no key gets O = 0 and L = -inf, and no other row does: where a score is NaN or
      // past fp32's range, l or m carries it (the maximum alone drops NaN), so neither is asked here.
      const bool sees = lim + item->j0 * BN > 0;
      float* part = p.parts + (size_t)(blockIdx.x * 2 + item->slot) * part_floats(D, ROWS);
      float m = m_run, l = l_run, f;
      if constexpr (SPLIT) {
        // A row's 2 REP states (two warpgroups, REP copies) become one. (m, l) are final before the
        // last product is: they meet here, so that O~ is scaled as it is read. The barrier also
        // says that the previous item's sums are done with the stage.
        float2* states = reinterpret_cast<float2*>(smem + LY::OFF_STATE);
        states[g * BM + r] = make_float2(m_run, l_run);
        if (!(ok = epi_sync())) break;
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int x = 0; x < 2 * REP; ++x) m = fmaxf(m, states[x * (BM / REP) + row].x);
        auto weight = [&](float mx) { return mx == -INFINITY ? 0.f : ex2_approx(mx - m); };
#pragma unroll
        for (int x = 0; x < 2 * REP; ++x) {
          const float2 st = states[x * (BM / REP) + row];
          l += st.y * weight(st.x);
        }
        f = weight(m_run);
      } else {
        f = 1.f;
      }
      // a whole item's O~ is divided by l; a partial state stays as it is
      if (!partial) f *= sees ? 1.f / l : 0.f;
      const int prow = SPLIT ? row : g * BM + row;
      const long long t = item->tok0 + tok;
      const int head = item->h * p.G + row_head;
      if (valid && (!SPLIT || (g == 0 && copy == 0))) {
        if (partial) *reinterpret_cast<float2*>(part + ROWS * D + 2 * prow) = make_float2(m, l);
        else if (p.L) p.L[t * (p.Hkv * p.G) + head] = sees ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
      if (worked) {
        ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->o_done[g]), o_ph, abort_flag, p));
        if (!ok) break;
        o_ph ^= 1;
        tc_fence_after();
      }
      if constexpr (!SPLIT) {
        // A warp's 32 rows leave through its own 4 KB of the stage, 128 bytes of each row at a time
        // (64 columns of O, 32 of a partial state), so that its stores are whole 128-byte lines: 16-byte
        // stores of 32 different rows took 5 us for an item's partial state (d = 128). 16-byte piece k
        // of row r stands at place k ^ (r & 7).
        const uint32_t mine = sStage + (uint32_t)warp * 4096u;
        const unsigned long long to = reinterpret_cast<unsigned long long>(
            partial ? (void*)(part + (size_t)prow * D)
                    : (void*)(p.o.ptr + t * p.o.ts + (long long)head * p.o.hs));
        const uint32_t live = __ballot_sync(0xffffffffu, valid);
        unsigned long long dsts[8];  // of the 8 rows that this lane sends pieces of
#pragma unroll
        for (int i = 0; i < 8; ++i) dsts[i] = __shfl_sync(0xffffffffu, to, 4 * i + (lane >> 3)) + (lane & 7) * 16;
        auto send = [&](int byte0) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // 4 rows at a time, 8 lanes each
            const int rr = 4 * i + (lane >> 3);
            uint32_t v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(mine + (uint32_t)rr * 128u + (uint32_t)(((lane & 7) ^ (rr & 7)) << 4))
                         : "memory");
            if (live >> rr & 1)
              *reinterpret_cast<uint4*>(dsts[i] + byte0) = make_uint4(v[0], v[1], v[2], v[3]);
          }
          __syncwarp();
        };
        auto put = [&](int k, uint32_t a, uint32_t b, uint32_t c4, uint32_t d4) {
          st_shared_v4(mine + (uint32_t)lane * 128u + (uint32_t)((k ^ (lane & 7)) << 4), a, b, c4, d4);
        };
        if (partial) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tO + q * 32, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int k = 0; k < 8; ++k) put(k, o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            send(q * 128);
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < D / 64; ++q) {
            uint32_t o[2][32];
            tmem_ld32(tO + q * 64, o[0]);
            tmem_ld32(tO + q * 64 + 32, o[1]);
            tmem_wait_ld();
            reg_fence(o[0]);
            reg_fence(o[1]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(o[k >> 2][8 * (k & 3) + e]) * f;
              const uint4 w16 = pack8<BF16>(x);
              put(k, w16.x, w16.y, w16.z, w16.w);
            }
            send(q * 128);
          }
        }
        tc_fence_before();
      } else {
        // All states of the item's rows side by side in the stage, row x R + row for state x; if
        // they are too many, half of the columns at a time. 16-byte piece i stands at i ^ (row & 7).
        const int R = item->nt * p.G, states_n = item->n > 1 ? 2 * REP : REP;  // (the second warpgroup's)
        const int srow = (g * REP + copy) * R + row;
        auto join = [&](auto cols_c, int col0) -> bool {
          constexpr int COLS = decltype(cols_c)::value;
          auto stage_at = [&](int rr, int i) { return sStage + (uint32_t)(rr * COLS * 4 + ((i ^ (rr & 7)) << 4)); };
          if (worked) {
#pragma unroll 1
            for (int q = 0; q < COLS; q += 64) {
              uint32_t o[2][32];
              tmem_ld32(tO + col0 + q, o[0]);
              tmem_ld32(tO + col0 + q + 32, o[1]);
              tmem_wait_ld();
              reg_fence(o[0]);
              reg_fence(o[1]);
              if (valid) {
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  const uint32_t* v = &o[k >> 3][4 * (k & 7)];
                  st_shared_v4(stage_at(srow, q / 4 + k), __float_as_uint(__uint_as_float(v[0]) * f),
                               __float_as_uint(__uint_as_float(v[1]) * f), __float_as_uint(__uint_as_float(v[2]) * f),
                               __float_as_uint(__uint_as_float(v[3]) * f));
                }
              }
              __syncwarp();
            }
            tc_fence_before();
          }
          if (!epi_sync()) return false;
          // sums over the states: thread = 4 columns of a row
#pragma unroll 1
          for (int x = threadIdx.x; x < R * (COLS / 4); x += 256) {
            const int rr = x / (COLS / 4), c4 = x % (COLS / 4);
            const int rt = token_of_row(p, rr);
            if (!storable(rt, rr - rt * p.G)) continue;
            float sum[4] = {};
#pragma unroll
            for (int a = 0; a < 2 * REP; ++a) {
              float y[4] = {};
              if (a < states_n) ld_shared_v4(stage_at(a * R + rr, c4), y);
#pragma unroll
              for (int e = 0; e < 4; ++e) sum[e] += y[e];
            }
            const int col = col0 + 4 * c4;
            if (partial) {
              *reinterpret_cast<float4*>(part + (size_t)rr * D + col) = make_float4(sum[0], sum[1], sum[2], sum[3]);
            } else {
              uint16_t* dst = p.o.ptr + (long long)(item->tok0 + rt) * p.o.ts +
                              (long long)(item->h * p.G + rr - rt * p.G) * p.o.hs + col;
              *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(sum[0], sum[1]), pack2<BF16>(sum[2], sum[3]));
            }
          }
          return true;
        };
        if (D == 64 || 2 * REP * R <= LY::STAGE_ROWS) {
          ok = join(std::integral_constant<int, D>{}, 0);
        } else if constexpr (D == 128) {
          ok = join(std::integral_constant<int, 64>{}, 0) && epi_sync() && join(std::integral_constant<int, 64>{}, 64);
        }
        if (!ok) break;
      }
      item_done();
    }
    tc_fence_before();
    named_bar_sync(1, NUM_THREADS);
  }
}

// Joins the partial states of the items that lie in several blocks' ranges: blocks (c, y) take the
// item that begins in block c's range. A warp joins RW rows at once, so that their loads overlap:
// lane = (row, piece) for the pieces' weights, then all lanes along the columns. (With no bound on the
// blocks the compiler saved registers by loading one piece after another: 100 tokens of 8 heads over 4000
// keys of one, d 128, 21.7 against 20.4 us, one sequence of 1001 keys 9.8 against 9.5.)
// Latency bounds it for single tokens; a chunk of 2048 tokens reads 37 MB of partial states (16.5 us
// with cold caches, 6 us for one token of one sequence).
template <int D, bool BF16, int ROWS>
__global__ void __launch_bounds__(COMBINE_THREADS, 4) fa_paged_combine_kernel(const __grid_constant__ Params p) {
  constexpr int E = D / 32;  // columns per lane
  constexpr int RW = ROWS > 128 ? 2 : 1, PB = 32 / RW;  // rows of a warp, pieces at a time
  launch_dependents();
  wait_previous_grid();
  const int4 rec0 = *reinterpret_cast<const int4*>(p.records + blockIdx.x * 8);
  const int4 rec1 = *reinterpret_cast<const int4*>(p.records + blockIdx.x * 8 + 4);
  if (rec0.x == 0) return;
  const int c0 = blockIdx.x, slot0 = rec0.y, n = rec0.z - c0 + 1, h = rec0.w, tok0 = rec1.x, nt = rec1.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, Hq = p.Hkv * p.G;
  if (!in_bounds(p, n > 1 && rec0.z < (int)gridDim.x && (c0 * 2 + slot0 + 1ll) * part_floats(D, ROWS) <= p.parts_len &&
                        (rec0.z * 2 + 1ll) * part_floats(D, ROWS) <= p.parts_len && tok0 >= 0 && tok0 + nt <= p.T &&
                        (h + 1) * p.G <= p.o.H))
    return;
  auto part = [&](int x) {  // piece x of the item
    return p.parts + (size_t)((c0 + x) * 2 + (x == 0 ? slot0 : 0)) * part_floats(D, ROWS);
  };
  const int pr0 = (blockIdx.y * (COMBINE_THREADS / 32) + warp) * RW;
  auto token_of = [&](int pr) {  // -1: the place holds no row
    const int row = pr % BM, tok = token_of_row(p, row) + pr / BM * p.tpt;
    return row < p.tpt * p.G && tok < nt ? tok : -1;
  };
  const int my_row = lane / PB, my_piece = lane % PB;
  const bool mine = token_of(pr0 + my_row) >= 0;
  auto state = [&](int x) {
    return mine && x < n ? *reinterpret_cast<const float2*>(part(x) + ROWS * D + 2 * (pr0 + my_row))
                         : make_float2(-INFINITY, 0.f);
  };
  const float2 st0 = state(my_piece);
  float m = st0.x;
  for (int x = my_piece + PB; x < n; x += PB) m = fmaxf(m, state(x).x);
#pragma unroll
  for (int o = PB / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[RW][E] = {}, l = 0.f;
  for (int x0 = 0; x0 < n; x0 += PB) {
    const float2 st = x0 == 0 ? st0 : state(x0 + my_piece);
    const float w = st.x != -INFINITY ? ex2_approx(st.x - m) : 0.f;
    l += st.y * w;
    const int k = min(PB, n - x0);
    // N pieces' rows in flight at once
    auto add = [&](auto n_c, int y) {
      constexpr int N = decltype(n_c)::value;
      float v[N][RW][E], wy[N][RW];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float* src = part(x0 + y + i) + (size_t)pr0 * D + lane * E;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          wy[i][r] = __shfl_sync(0xffffffffu, w, r * PB + y + i);
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][r][e] = 0.f;
          if (wy[i][r] != 0.f) {
            if constexpr (E == 4) {
              const float4 q = *reinterpret_cast<const float4*>(src + r * D);
              v[i][r][0] = q.x, v[i][r][1] = q.y, v[i][r][2] = q.z, v[i][r][3] = q.w;
            } else {
              const float2 q = *reinterpret_cast<const float2*>(src + r * D);
              v[i][r][0] = q.x, v[i][r][1] = q.y;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[r][e] = fmaf(v[i][r][e], wy[i][r], acc[r][e]);
    };
    int y = 0;
#pragma unroll 1
    for (; y + 4 <= k; y += 4) add(std::integral_constant<int, 4>{}, y);
    if (y + 2 <= k) add(std::integral_constant<int, 2>{}, y), y += 2;
    if (y < k) add(std::integral_constant<int, 1>{}, y);
  }
#pragma unroll
  for (int o = PB / 2; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const float lr = __shfl_sync(0xffffffffu, l, r * PB), mr = __shfl_sync(0xffffffffu, m, r * PB);
    const int tok = token_of(pr0 + r);
    if (tok < 0) continue;
    const bool sees = rec1.z + (p.causal ? tok : 0) > 0;  // as in the main kernel; a piece's NaN is in its l
    const float inv = sees ? 1.f / lr : 0.f;
    const long long t = tok0 + tok;
    const int head = h * p.G + (pr0 + r) % BM % p.G;
    uint16_t* dst = p.o.ptr + t * p.o.ts + (long long)head * p.o.hs + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack2<BF16>(acc[r][e] * inv, acc[r][e + 1] * inv);
    if (p.L && lane == 0) p.L[t * Hq + head] = sees ? (mr + log2f(lr)) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace paged
}  // namespace fa
