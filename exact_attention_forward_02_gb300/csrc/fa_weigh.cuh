// fa_weigh.cuh -- the attention weight that the new tokens of each sequence give to every cached token.
// Included by fa_evict.cu.
//
//   w_j = (w_j of before, for tokens that are not new) + sum over the rows i that see j of exp(scale <q_i, k_j> - L_i)
// for every key head, over the rows of all its query heads; L is what the attention returned.
//
// Products are transposed, S^T = K Q^T: a tile of 128 keys is the left operand (TMEM lane = thread = key)
// and rows of q are the columns, so that a key's weight is a sum along the thread's own columns: no
// exchange between threads, no atomics, one order of summation. A unit is (sequence, key head, 256 keys):
// its two key tiles stay in shared memory, one to each softmax warpgroup, while tiles of up to 128 rows
// of q go by. Units are shared out to the SMs from the lengths on the device, by cost. With a causal mask
// later keys are seen by fewer rows: a head's units are dealt from both ends in turn, so that any run of
// them costs about its share.
//
// Three forms, by the cache and the rows (MODE):
//   HALF    a 16-bit cache
//   TURNED  a cache in 8 bits, more than 16 rows: 4 more warps turn each key tile into the type of q, exactly, once
//           for all rows
//   HELD    a cache in 8 bits, up to 16 rows (single tokens, drafts): the products take K as it is held, and a warp
//           splits the rows into sums of E4M3 numbers (split_row), side by side as columns; turning K would cost
//           shared memory as many cycles as HBM takes to bring it (fa_paged.cuh)
// A key's scale is its thread's own factor. 12 warps and those: 0-7 softmax, 8 and 11 loads (a key tile each, pages
// box by box), 9 MMA issuer. Single tokens are bound by HBM (K is read once), chunks by the tensor cores and the
// exponentials, which take the same time (128 x 128 scores: 545 and 512 cycles). Neither is reached: a unit of few rows
// takes 2600 cycles where its bytes take 1400, the chain from its keys to its sums (64 ragged sequences, 8 key heads,
// d 128, pages of 16: 81 us in 8 bits, 3.6 TB/s, 94 in 16, 6.0 TB/s), and a chunk is held up by that chain and by 256
// units for 152 SMs (2048 tokens at 30720, Hq 16, Hkv 2, d 128: 304 us, 0.87 PFLOP/s, tensor pipe 35 %).
#pragma once

#include "fa_paged.cuh"

namespace fa {
namespace weigh {

using paged::BM;
using paged::BN;
using paged::wait_compact;
using paged::wait_drain;
enum Mode { HALF, TURNED, HELD };
constexpr int HELD_ROWS = 16;
constexpr int WARP_LOAD = 8, WARP_MMA = 9, WARP_LOAD2 = 11, WARP_CONVERT = 12;
constexpr int MAX_SLOTS = 4;
constexpr int COST_UNIT = 2;  // what a unit costs beside its row tiles, in those

struct Params {
  const float* L;
  const float* ks;  // F8: scales [num_pages][Hkv]
  float* w;         // [num_pages][Hkv][page_size]
  HeadsDev q;       // HELD
  int num_pages, page_size, page_shift, box_keys;  // page_shift: log2 of the page size, -1 where that is none
  int Hkv, G, Hq, tpt, cols;  // tpt: tokens per tile of rows; cols = tpt G
  uint32_t by_g;              // ceil(2^16 / G)
  const int *cu, *lens, *table;
  int table_stride, B, T, causal, cap;
  float c;  // scale * log2(e)
  unsigned long long wait_limit_ns;
  int* status;
};

struct Barriers {
  uint64_t q_full[4], q_empty[4];
  uint64_t k_full[2][MAX_SLOTS], k_empty[2][MAX_SLOTS];  // [key tile of a unit]
  uint64_t raw_full[2][MAX_SLOTS], raw_empty[2][MAX_SLOTS];
  uint64_t s_full[2][2], s_empty[2][2];
  uint64_t paused;  // the second warpgroup has read all it wants, and the next unit has one key tile
  uint64_t mma_drain;
  long long warp_cost[16];
  long long start_rem;
  int start_b;
  uint32_t tmem_base;
  int abort_flag;
};

template <int D, bool BF16, int MODE>
struct Layout {
  static constexpr int TERMS = BF16 ? 2 : 3, NQ = TERMS * HELD_ROWS;  // HELD: columns, term by term
  static constexpr int CHUNK_BYTES = BM * 128, CHUNKS = D / 64;
  // tiles that the products read, and tiles as they are loaded where they have to be turned
  static constexpr int TILE_BYTES = MODE == HELD ? BM * D : BM * D * 2, RAW_BYTES = BM * D;
  static constexpr int Q_BYTES = MODE == HELD ? NQ * D : BM * D * 2;
  static constexpr int Q_SLOTS = D == 64 || MODE == HELD ? 4 : 2;
  // slots of each of a unit's two key tiles, which have rings of their own: a unit may have one tile only, and a ring
  // shared by two loading warps would pass the one that has nothing to load
  static constexpr int K_SLOTS = MODE == HELD ? 4 : D == 64 ? (MODE == TURNED ? 2 : 3) : (MODE == TURNED ? 1 : 2);
  static constexpr int RAW_SLOTS = MODE != TURNED ? 0 : D == 64 ? 3 : 2, RAW_RING = MODE == TURNED ? RAW_SLOTS : 1;
  static constexpr int S_COLS = MODE == HELD ? 64 : 128;  // of one of the four buffers of S^T
  static constexpr int OFF_Q = 0, OFF_K = (Q_SLOTS * Q_BYTES + 1023) / 1024 * 1024, OFF_RAW = OFF_K + 2 * K_SLOTS * TILE_BYTES;
  // -L log2 e of the rows, of eight tiles of them, and with HELD their 2^e
  static constexpr int L_ROWS = MODE == HELD ? HELD_ROWS : BM;
  static constexpr int OFF_L = OFF_RAW + 2 * RAW_SLOTS * RAW_BYTES;
  static constexpr int OFF_EXP = OFF_L + 8 * L_ROWS * 4;
  static constexpr int OFF_BAR = OFF_EXP + (MODE == HELD ? 8 * HELD_ROWS * 4 : 0);
  static constexpr int SMEM_BYTES = OFF_BAR + 1024;
  static_assert(sizeof(Barriers) <= 1024 && SMEM_BYTES <= paged::SMEM_LIMIT, "shared memory budget");
};

struct Seq {
  int t0, n, len, units;  // first row of q, new tokens, cached tokens, units of a head
  int cost, qn;           // of a unit; tiles of rows
};
struct Unit {
  int b, h, t0, n, len, key0, q0, qn;  // first key; tiles of rows [q0, qn) see one of its keys
  bool two;                            // its second key tile holds a key
  bool same;                           // its one tile of rows is that of the unit before
};

__device__ __forceinline__ Seq load_seq(const Params& p, int b, bool report) {
  Seq s;
  s.t0 = p.cu[b];
  const int end = p.cu[b + 1], len = p.lens[b];
  const bool rows_ok = s.t0 >= 0 && end >= s.t0 && end <= p.T;
  s.n = rows_ok ? end - s.t0 : 0;
  s.len = s.n ? max(0, min(len, p.cap)) : 0;
  s.units = (int)(((uint32_t)s.len + 255u) / 256u);
  const int qt = s.n <= p.tpt ? (s.n > 0) : (s.n - 1) / p.tpt + 1;
  s.qn = qt;
  s.cost = COST_UNIT + qt;
  if (p.causal && s.len) {  // rows see the new keys in part
    const long long seen = 2ll * s.len - min(s.n, s.len);
    s.cost = COST_UNIT + (int)((qt * seen + 2ll * s.len - 1) / (2ll * s.len));
  }
  if (report && (!rows_ok || (s.n && len > p.cap))) atomicCAS(p.status, 0, FA_ERR_RANGE);
  return s;
}

// Walks a block's units; every role does so by itself.
struct Walk {
  Seq s;
  int b, idx;  // unit of the sequence: head * units + place
  int h, i;    // those two
  bool one;    // the last unit had one tile of rows, the first
  long long u, u1;
  __device__ __forceinline__ void begin(const Params& p, const Barriers* bars, long long u0, long long end) {
    u1 = end;
    u = u0;
    b = bars->start_b;
    idx = 0;
    s = Seq{};
    h = i = 0;
    one = false;
    if (u0 >= u1) return;
    s = load_seq(p, b, false);
    // the first unit that begins in the range
    const long long skip = (bars->start_rem + s.cost - 1) / s.cost;
    idx = (int)skip;
    u += skip * s.cost - bars->start_rem;
    if (idx < p.Hkv * s.units) {
      h = idx / s.units;
      i = idx - h * s.units;
    }
  }
  __device__ __forceinline__ bool next(const Params& p, Unit& x) {
    while (u < u1) {
      if (idx < p.Hkv * s.units) {
        const int j = i & 1 ? s.units - 1 - (i >> 1) : i >> 1;
        x.b = b;
        x.h = h;
        x.t0 = s.t0;
        x.n = s.n;
        x.len = s.len;
        x.key0 = j * 256;
        x.q0 = p.causal && s.qn > 1 && x.key0 > s.len - s.n ? (x.key0 - (s.len - s.n)) / p.tpt : 0;
        x.qn = s.qn;
        x.two = s.len - x.key0 > BN;
        x.same = one && x.qn == 1;
        one = x.qn == 1;
        ++idx;
        u += s.cost;
        if (++i == s.units) i = 0, ++h, one = false;
        return true;
      }
      do {
        if (++b >= p.B) return false;
        s = load_seq(p, b, false);
      } while (s.units == 0);
      idx = h = i = 0;
      one = false;
    }
    return false;
  }
};

__host__ __device__ constexpr int num_warps(int mode) { return mode == TURNED ? 16 : mode == HELD ? 13 : 12; }

template <int D, bool BF16, int MODE>
__global__ void __launch_bounds__(num_warps(MODE) * 32, 1)
    fa_weigh_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ Params p) {
  using LY = Layout<D, BF16, MODE>;
  constexpr int NUM_WARPS = num_warps(MODE), NUM_THREADS = NUM_WARPS * 32;
  constexpr bool F8 = MODE != HALF;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, FA_ERR_ALIGN);
    return;
  }
  Barriers* bars = reinterpret_cast<Barriers*>(smem + LY::OFF_BAR);
  const uint32_t sQ = smem_u32(smem + LY::OFF_Q), sK = smem_u32(smem + LY::OFF_K), sRaw = smem_u32(smem + LY::OFF_RAW);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < LY::Q_SLOTS; ++s) {
      mbar_init(smem_u32(&bars->q_full[s]), 1);
      mbar_init(smem_u32(&bars->q_empty[s]), 1);
    }
    for (int s = 0; s < LY::K_SLOTS; ++s) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(smem_u32(&bars->k_full[x][s]), MODE == TURNED ? 4 : 1);
        mbar_init(smem_u32(&bars->k_empty[x][s]), 1);
      }
    }
    for (int s = 0; s < LY::RAW_SLOTS; ++s) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(smem_u32(&bars->raw_full[x][s]), 1);
        mbar_init(smem_u32(&bars->raw_empty[x][s]), 4);
      }
    }
    for (int x = 0; x < 4; ++x) {
      mbar_init(smem_u32(&bars->s_full[x >> 1][x & 1]), 1);
      mbar_init(smem_u32(&bars->s_empty[x >> 1][x & 1]), 4);
    }
    mbar_init(smem_u32(&bars->paused), 4);
    mbar_init(smem_u32(&bars->mma_drain), 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == WARP_LOAD && lane == 0) {
    if (MODE != HELD) tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
  }
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  launch_dependents();
  wait_previous_grid();  // no global memory is read or written before this
  tc_fence_before();
  // The block's share [u0, u1) of all units' costs, and the sequence that u0 lies in.
  long long u0, u1;
  {
    const int per_thread = (p.B + NUM_THREADS - 1) / NUM_THREADS;
    const int b0 = min((int)threadIdx.x * per_thread, p.B), b1 = min(b0 + per_thread, p.B);
    auto cost_of = [&](int b, bool report) -> long long {
      const Seq s = load_seq(p, b, report);
      return (long long)p.Hkv * s.units * s.cost;
    };
    long long mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += cost_of(b, blockIdx.x == 0);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) bars->warp_cost[warp] = incl;
    __syncthreads();
    long long before = incl - mine, W = 0;
#pragma unroll
    for (int w = 0; w < NUM_WARPS; ++w) {
      if (w < warp) before += bars->warp_cost[w];
      W += bars->warp_cost[w];
    }
    u0 = paged::divide((long long)blockIdx.x * W, (int)gridDim.x);
    u1 = paged::divide((blockIdx.x + 1ll) * W, (int)gridDim.x);
    if (u0 < u1 && before <= u0 && u0 < before + mine) {
      int b = b0;
#pragma unroll 1
      for (; b + 1 < b1; ++b) {
        const long long x = cost_of(b, false);
        if (u0 < before + x) break;
        before += x;
      }
      bars->start_b = b;
      bars->start_rem = u0 - before;
    }
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  Walk walk;
  walk.begin(p, bars, u0, u1);
  Unit it;
  auto wait_all = [&](uint64_t* bar, uint32_t par) -> bool {
    return __all_sync(0xffffffffu, wait_compact(smem_u32(bar), par, abort_flag, p));
  };
  // L of column `col` of a tile of rows, in base 2 and negative; 0 for a column without a row
  auto ask_row = [&](const Unit& u, int q, int col) {
    const int tok = (int)((uint32_t)col * p.by_g >> 16), t = q * p.tpt + tok;
    return col < p.cols && t < u.n ? p.L[(size_t)(u.t0 + t) * p.Hq + u.h * p.G + col - tok * p.G] * -1.4426950408889634f : 0.f;
  };
  // Whoever brings tile m of the rows writes what belongs to them when the products of tile m - Q_SLOTS are done. The last
  // of those were issued when the warpgroup's scores of the product but two before had been read, so it may still look
  // at what belongs to tile m - Q_SLOTS - 2 and on, and there is room for eight. The second warpgroup has no part in
  // units of one key tile, however many: before rows are brought for those, it has read all that its own last product
  // wants (paused; s_empty says only that scores have been read).
  auto page_of = [&](int key) { return p.page_shift >= 0 ? (uint32_t)key >> p.page_shift : (uint32_t)key / (uint32_t)p.page_size; };

  if (warp == WARP_LOAD || warp == WARP_LOAD2) {
    // ========================================================================= loads
    // Key tile x of a unit (x: the warp) goes box by box, a page each; warp 8 loads the rows of q as well. Table
    // entries are asked for a unit ahead.
    const int x = warp == WARP_LOAD2;
    constexpr int BOX_CHUNKS = F8 ? 1 : LY::CHUNKS, SLOTS = MODE == TURNED ? LY::RAW_SLOTS : LY::K_SLOTS;
    constexpr uint32_t BOX_ROW = F8 ? D : 128, SLOT_BYTES = MODE == TURNED ? LY::RAW_BYTES : LY::TILE_BYTES;
    uint64_t* const full = MODE == TURNED ? bars->raw_full[x] : bars->k_full[x];
    uint64_t* const empty = MODE == TURNED ? bars->raw_empty[x] : bars->k_empty[x];
    const uint32_t sLoad = (MODE == TURNED ? sRaw : sK) + x * SLOTS * SLOT_BYTES;
    const int box_shift = 31 - __clz(p.box_keys), boxes = BN >> box_shift, my_box = lane & (boxes - 1);
    const int my_chunk = lane / boxes;
    const uint32_t box_bytes = (uint32_t)p.box_keys * BOX_ROW;
    const uint32_t box_off = (uint32_t)my_chunk * LY::CHUNK_BYTES + (uint32_t)my_box * box_bytes;
    const uint32_t q_bytes = (uint32_t)(LY::CHUNKS * p.cols) * 128u;
    uint32_t slot = 0, par = 0, nq = 0, k_mask = 0, k_par = 0;  // par: uses of the ring so far, as a parity
    uint32_t used = 0;                                          // key tiles so far, up to SLOTS
    bool ok = true;
    auto entry = [&](const Unit& u) -> int {  // of the lane's box
      const int key = u.key0 + x * BN + (my_box << box_shift);
      return key < u.len ? p.table[(size_t)u.b * p.table_stride + page_of(key)] : 0;
    };
    bool have = walk.next(p, it);
    int page = have ? entry(it) : 0;
    while (ok && have) {
      Unit nx;
      const bool more = walk.next(p, nx);
      const int next_page = more ? entry(nx) : 0;
      const int key = it.key0 + x * BN + (my_box << box_shift);
      if (key < it.len && (page < 0 || page >= p.num_pages)) {
        atomicCAS(p.status, 0, FA_ERR_RANGE);
        page = p.num_pages;  // reads as zeros
      }
      if (x == 0 || it.two) {
        if (used == SLOTS) ok = wait_all(&empty[slot], par ^ 1u);
        else ++used;
        if (!ok) break;
        const int keys = it.len - it.key0 - x * BN;
        const int live = min(boxes, (keys + p.box_keys - 1) >> box_shift);
        const uint32_t bar = smem_u32(&full[slot]);
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(live * BOX_CHUNKS) * box_bytes);
        __syncwarp();
        in_bounds(p, my_chunk >= BOX_CHUNKS || my_box >= live || (it.h < p.Hkv && page >= 0 && page <= p.num_pages));
        if (my_chunk < BOX_CHUNKS && my_box < live)
          tma_load_4d(sLoad + slot * SLOT_BYTES + box_off, &tmK, bar, my_chunk * 64, p.page_size > BN ? key % p.page_size : 0,
                      it.h, page);
        k_mask |= 1u << slot;
        k_par = (k_par & ~(1u << slot)) | (par << slot);
        if (++slot == SLOTS) slot = 0, par ^= 1u;
      }
      if (MODE != HELD && x == 0 && !it.same) {
#pragma unroll 1
        for (int q = it.q0; q < it.qn && ok; ++q, ++nq) {
          const uint32_t qs = nq % LY::Q_SLOTS, round = nq / LY::Q_SLOTS;
          float l4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) l4[i] = ask_row(it, q, lane * 4 + i);
          if (round > 0 && !(ok = wait_all(&bars->q_empty[qs], (round - 1) & 1u))) break;
          *reinterpret_cast<float4*>(smem + LY::OFF_L + ((nq & 7u) * LY::L_ROWS + lane * 4) * 4) = make_float4(l4[0], l4[1], l4[2], l4[3]);
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(smem_u32(&bars->q_full[qs]), q_bytes);
          __syncwarp();
          in_bounds(p, it.t0 >= 0 && it.t0 + q * p.tpt < p.T && (it.h + 1) * p.G <= p.Hq);
          if (lane < LY::CHUNKS)
            tma_load_3d(sQ + qs * LY::Q_BYTES + lane * LY::CHUNK_BYTES, &tmQ, smem_u32(&bars->q_full[qs]), lane * 64,
                        it.h * p.G, it.t0 + q * p.tpt);
        }
      }
      it = nx;
      page = next_page;
      have = more;
    }
    if (!ok && lane == 0) {  // every issued copy must land before the block may exit
      for (int s = 0; s < SLOTS; ++s)
        if (k_mask & (1u << s)) wait_drain(smem_u32(&full[s]), (k_par >> s) & 1u, p);
      for (uint32_t q = nq > LY::Q_SLOTS ? nq - LY::Q_SLOTS : 0; x == 0 && q < nq; ++q)
        wait_drain(smem_u32(&bars->q_full[q % LY::Q_SLOTS]), (q / LY::Q_SLOTS) & 1u, p);
    }
    __syncwarp();
  } else if (warp == WARP_MMA) {
    // ========================================================================= MMA issuer
    constexpr uint64_t SW = MODE == HELD && D == 64 ? UMMA_SWIZZLE_64B : UMMA_SWIZZLE_128B;
    constexpr uint32_t SBO = MODE == HELD && D == 64 ? 512 : 1024;
    const uint32_t id = MODE == HELD ? umma_idesc_f16(0, 0, 0, BM, LY::NQ)
                                     : umma_idesc_f16(BF16 ? 1 : 0, 0, 0, BM, (uint32_t)(p.cols + 15) / 16 * 16);
    const uint64_t dQ = umma_smem_desc<SW>(sQ, 16, SBO), dK = umma_smem_desc<SW>(sK, 16, SBO);
    uint32_t ks[2] = {0, 0}, k_par[2] = {0, 0}, nq = 0;  // places in K's rings; tiles of rows so far
    uint32_t sn[2] = {0, 0};                             // products of each warpgroup
    // A pause of the second warpgroup is waited for when other rows come, or before its next product, so that its
    // barrier is never a phase ahead.
    bool pause = false, two = false;
    uint32_t pauses = 0;
    bool ok = true;
    auto ok_pause = [&]() {
      if (pause) ok = wait_all(&bars->paused, pauses++ & 1u);
      pause = false;
      return ok;
    };
    while (ok && walk.next(p, it)) {
      const int tiles = it.two ? 2 : 1;
      if (it.two && !ok_pause()) break;
      pause = pause || (two && !it.two);
      two = it.two;
#pragma unroll 1
      for (int q = it.q0; q < it.qn && ok; ++q) {
        if (!it.same) {  // the rows of before are given back when others come
          if (nq && elect_one()) umma_commit(smem_u32(&bars->q_empty[(nq - 1) % LY::Q_SLOTS]));
          __syncwarp();
          if (!ok_pause()) break;
          if (!(ok = wait_all(&bars->q_full[nq % LY::Q_SLOTS], (nq / LY::Q_SLOTS) & 1u))) break;
          ++nq;
        }
        const uint64_t db = dQ + (((nq - 1) % LY::Q_SLOTS * LY::Q_BYTES) >> 4);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x >= tiles) break;
          const uint32_t n = sn[x]++, buf = n & 1u;
          if (q == it.q0 && !(ok = wait_all(&bars->k_full[x][ks[x]], k_par[x]))) break;
          if (!(ok = wait_all(&bars->s_empty[x][buf], ((n >> 1) & 1u) ^ 1u))) break;
          tc_fence_after();
          const uint64_t da = dK + (((x * LY::K_SLOTS + ks[x]) * LY::TILE_BYTES) >> 4);
          const uint32_t to = tmem + x * 256 + buf * LY::S_COLS;
          if (elect_one()) {
            if constexpr (MODE == HELD) {
#pragma unroll
              for (int k = 0; k < D / 32; ++k) umma_ss_f8(to, da + (k * 32 >> 4), db + (k * 32 >> 4), id, k > 0 ? 1u : 0u);
            } else {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k >> 2) * LY::CHUNK_BYTES + (k & 3) * 32) >> 4;
                umma_ss(to, da + off, db + off, id, k > 0 ? 1u : 0u);
              }
            }
            umma_commit(smem_u32(&bars->s_full[x][buf]));
            if (q + 1 == it.qn) umma_commit(smem_u32(&bars->k_empty[x][ks[x]]));
          }
          __syncwarp();
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (x < tiles && ++ks[x] == LY::K_SLOTS) ks[x] = 0, k_par[x] ^= 1u;
    }
    if (elect_one()) umma_commit(smem_u32(&bars->mma_drain));
    __syncwarp();
    wait_drain(smem_u32(&bars->mma_drain), 0, p);
    __syncwarp();
  } else if (MODE == HELD && warp >= WARP_CONVERT) {
    // ========================================================================= rows split
    constexpr int QL = D / 8, Q_TURN = 32 / QL, TERMS = LY::TERMS;  // lanes of a row, rows at a time
    const int ql = lane % QL;
    float* exps = reinterpret_cast<float*>(smem + LY::OFF_EXP);
    uint32_t nq = 0;
    bool ok = true;
    while (ok && walk.next(p, it)) {
      if (it.same) continue;
#pragma unroll 1
      for (int q = it.q0; q < it.qn && ok; ++q, ++nq) {
        const uint32_t qs = nq % LY::Q_SLOTS, round = nq / LY::Q_SLOTS;
        const int rows = min(p.tpt, it.n - q * p.tpt) * p.G;
        auto load = [&](int r) {  // (zeros where there is no row)
          const int tok = (int)((uint32_t)r * p.by_g >> 16);
          if (r >= rows || !in_bounds(p, it.t0 >= 0 && it.t0 + q * p.tpt + tok < p.T && it.h * p.G + r - tok * p.G < p.q.H))
            return make_uint4(0, 0, 0, 0);
          return *reinterpret_cast<const uint4*>(p.q.ptr + (long long)(it.t0 + q * p.tpt + tok) * p.q.ts +
                                                 (long long)(it.h * p.G + r - tok * p.G) * p.q.hs + ql * 8);
        };
        uint4 u = load(lane / QL);
        const float l = ask_row(it, q, lane);
        if (round > 0 && !(ok = wait_all(&bars->q_empty[qs], (round - 1) & 1u))) break;
#pragma unroll 1
        for (int r = lane / QL; r < HELD_ROWS; r += Q_TURN) {
          const uint4 next = load(r + Q_TURN);
          uint32_t w[TERMS][2];
          const int ex = paged::split_row<D, BF16>(u, w);
          u = next;
          if (ql == 0) exps[(nq & 7u) * HELD_ROWS + r] = __uint_as_float((uint32_t)(127 + ex) << 23);
          const uint32_t sw = D == 128 ? r & 7u : (r >> 1) & 3u;
#pragma unroll
          for (int m = 0; m < TERMS; ++m)
            st_shared_v2(sQ + qs * LY::Q_BYTES + (m * HELD_ROWS + r) * D + ((((uint32_t)ql >> 1) ^ sw) << 4) + (ql & 1) * 8,
                         w[m][0], w[m][1]);
        }
        if (lane < HELD_ROWS) *reinterpret_cast<float*>(smem + LY::OFF_L + ((nq & 7u) * HELD_ROWS + lane) * 4) = l;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->q_full[qs]));
      }
    }
  } else if (MODE == TURNED && warp >= WARP_CONVERT) {
    // ========================================================================= 8 bits to 16
    // Thread = 16 elements of a row at a time, as in fa_paged.cuh; behind the last key anything may stand.
    const int ct = (int)threadIdx.x - WARP_CONVERT * 32;
    constexpr int PIECES = D / 16, TURNS = PIECES, BATCH = 4;
    const int c16 = ct % PIECES, row0 = (ct / PIECES) ^ (c16 >> 2);
    const uint32_t half = (uint32_t)(c16 >> 2) * LY::CHUNK_BYTES, j0 = (c16 & 3) * 2;
    uint32_t n[2] = {0, 0};  // tiles so far
    bool ok = true;
    while (ok && walk.next(p, it)) {
#pragma unroll 1
      for (int x = 0; x < (it.two ? 2 : 1) && ok; ++x) {
        const uint32_t t = x ? n[1]++ : n[0]++;
        const uint32_t hs = t % LY::RAW_RING, ks = t % LY::K_SLOTS, round = t / LY::K_SLOTS;
        ok = wait_all(&bars->raw_full[x][hs], (t / LY::RAW_RING) & 1u);
        if (ok && round > 0) ok = wait_all(&bars->k_empty[x][ks], (round - 1) & 1u);
        if (!ok) break;
        const uint32_t from = sRaw + (x * LY::RAW_SLOTS + hs) * LY::RAW_BYTES + (uint32_t)(row0 * D + c16 * 16);
        const uint32_t to = sK + (x * LY::K_SLOTS + ks) * LY::TILE_BYTES + half;
#pragma unroll 1
        for (int y0 = 0; y0 < TURNS; y0 += BATCH) {
          uint32_t v[BATCH][4];
#pragma unroll
          for (int y = 0; y < BATCH; ++y) ld_shared_u4(from + (y0 + y) * 2048u, v[y]);
#pragma unroll
          for (int y = 0; y < BATCH; ++y) {
            const uint32_t row = (uint32_t)(row0 + (y0 + y) * (128 / PIECES));
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              unpack4_e4m3(v[y][e], w[2 * e], w[2 * e + 1]);
              if (BF16) {  // 4 of fp16's 11 bits are in use, and bf16 has 8
                float a, b;
                unpack2<false>(w[2 * e], a, b);
                w[2 * e] = pack2<true>(a, b);
                unpack2<false>(w[2 * e + 1], a, b);
                w[2 * e + 1] = pack2<true>(a, b);
              }
            }
            const uint32_t base = to + row * 128u, sw = row & 7u;
            st_shared_v4(base + ((j0 ^ sw) << 4), w[0], w[1], w[2], w[3]);
            st_shared_v4(base + (((j0 + 1) ^ sw) << 4), w[4], w[5], w[6], w[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars->k_full[x][ks]));
          mbar_arrive(smem_u32(&bars->raw_empty[x][hs]));
        }
      }
    }
  } else if (warp < 8) {
    // ========================================================================= softmax
    const int g = warp >> 2, wq = warp & 3;
    const uint32_t tS = tmem + ((uint32_t)(wq * 32) << 16) + g * 256;
    constexpr int CH = MODE == HELD ? 8 : 32;  // columns at a time
    const int chunks = (p.cols + CH - 1) / CH;
    // The thread's key in a unit: place of its weight, found two units ahead, so that its table entry, and then
    // its weight and scale, are there in time.
    struct Place {
      int page;
      uint32_t off;   // in the page's weights, which are fewer than 2^32
      bool held, old; // a cached token; not a new one
    };
    auto place_of = [&](const Unit& u) {
      Place x;
      const int key = u.key0 + g * BN + wq * 32 + lane;
      const uint32_t entry = page_of(key);
      x.held = key < u.len;
      x.old = key < u.len - u.n;
      x.page = x.held ? p.table[(size_t)u.b * p.table_stride + entry] : -1;
      x.off = (uint32_t)u.h * (uint32_t)p.page_size + ((uint32_t)key - entry * (uint32_t)p.page_size);
      return x;
    };
    auto weight_at = [&](const Place& x) { return p.w + (size_t)x.page * p.Hkv * p.page_size + x.off; };
    auto fetch = [&](Place& x, int h, float& w, float& k) {
      if (x.held && (x.page < 0 || x.page >= p.num_pages)) x.held = false;  // (reported by the loading warps)
      w = x.held && x.old ? *weight_at(x) : 0.f;
      k = F8 && x.held ? p.ks[(size_t)x.page * p.Hkv + h] : 1.f;
    };
    Unit nx, ny;
    bool have = walk.next(p, it), more = have && walk.next(p, nx), most = more && walk.next(p, ny);
    Place here = {}, then = {}, last = {};
    float w_here = 0.f, k_here = 1.f, w_then = 0.f, k_then = 1.f;
    if (have) here = place_of(it);
    if (more) then = place_of(nx);
    if (have) fetch(here, it.h, w_here, k_here);
    uint32_t sn = 0, nq = 0;
    bool ok = true;
    while (ok && have) {
      if (most) last = place_of(ny);
      if (more) fetch(then, nx.h, w_then, k_then);
      const bool mine = g == 0 || it.two;
      const int key = it.key0 + g * BN + wq * 32 + lane, ctx = it.len - it.n;
      const float ct = p.c * k_here;
      const uint64_t c2 = f2(ct, ct);
      uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll 1
      for (int q = it.q0; q < it.qn; ++q) {
        if (!it.same) ++nq;
        if (!mine) continue;
        const uint32_t buf = sn & 1u, from = tS + buf * LY::S_COLS;
        ok = wait_all(&bars->s_full[g][buf], (sn >> 1) & 1u);
        if (!ok) break;
        ++sn;
        tc_fence_after();
        const uint32_t sL = smem_u32(smem + LY::OFF_L) + ((nq - 1) & 7u) * (LY::L_ROWS * 4);
        // columns [lo, hi) are rows that see the thread's key
        const int hi = min(p.tpt, it.n - q * p.tpt) * p.G;
        const int lo = p.causal ? min(max(key - ctx - q * p.tpt, 0), p.tpt) * p.G : 0;
        auto done = [&](int x) {  // the scores are read
          if (x < chunks - 1) return;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->s_empty[g][buf]));
        };
        if constexpr (MODE == HELD) {
          const uint32_t sE = smem_u32(smem + LY::OFF_EXP) + ((nq - 1) & 7u) * (HELD_ROWS * 4);
#pragma unroll 1
          for (int x = 0; x < chunks; ++x) {
            uint32_t s[LY::TERMS][8];
#pragma unroll
            for (int m = 0; m < LY::TERMS; ++m) tmem_ld8(from + m * HELD_ROWS + x * 8, s[m]);
            tmem_wait_ld();
#pragma unroll
            for (int m = 0; m < LY::TERMS; ++m) reg_fence(s[m]);
            done(x);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float l4[4], e4[4], y[4];
              ld_shared_v4(sL + x * 32 + k * 16, l4);
              ld_shared_v4(sE + x * 32 + k * 16, e4);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float sum = __uint_as_float(s[LY::TERMS - 1][4 * k + i]);  // small ones first
#pragma unroll
                for (int m = LY::TERMS - 2; m >= 0; --m) sum += __uint_as_float(s[m][4 * k + i]);
                const int col = 8 * x + 4 * k + i;
                y[i] = ex2_approx(fmaf(sum * e4[i], ct, l4[i]));
                y[i] = col >= lo && col < hi ? y[i] : 0.f;
              }
              acc[2 * k] = f2_add(acc[2 * k], f2(y[0], y[1]));
              acc[2 * k + 1] = f2_add(acc[2 * k + 1], f2(y[2], y[3]));
            }
          }
        } else {
          auto add = [&](const uint32_t (&s)[32], int x, auto whole) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float l4[4], e[4];
              ld_shared_v4(sL + x * 128 + k * 16, l4);
              f2_split(f2_fma(f2(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1])), c2, f2(l4[0], l4[1])), e[0], e[1]);
              f2_split(f2_fma(f2(__uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3])), c2, f2(l4[2], l4[3])), e[2], e[3]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                e[i] = ex2_approx(e[i]);
                if (!decltype(whole)::value) e[i] = 32 * x + 4 * k + i >= lo && 32 * x + 4 * k + i < hi ? e[i] : 0.f;
              }
              acc[(2 * k) & 3] = f2_add(acc[(2 * k) & 3], f2(e[0], e[1]));
              acc[(2 * k + 1) & 3] = f2_add(acc[(2 * k + 1) & 3], f2(e[2], e[3]));
            }
          };
          const bool whole = __all_sync(0xffffffffu, lo == 0 && hi >= 32 * chunks);
#pragma unroll 1
          for (int x = 0; x < chunks; ++x) {
            uint32_t s[32];
            tmem_ld32(from + x * 32, s);
            tmem_wait_ld();
            reg_fence(s);
            done(x);
            if (whole) add(s, x, std::true_type{});
            else add(s, x, std::false_type{});
          }
        }
      }
      if (!ok) break;
      if (g == 1 && mine && more && !nx.two) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->paused));
      }
      if (mine && here.held && in_bounds(p, here.page >= 0 && here.page < p.num_pages && it.h < p.Hkv &&
                                                here.off / (uint32_t)p.page_size == (uint32_t)it.h)) {
        float a, b;
        f2_split(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a, b);
        *weight_at(here) = w_here + (a + b);
      }
      here = then;
      then = last;
      w_here = w_then;
      k_here = k_then;
      it = nx;
      nx = ny;
      have = more;
      more = most;
      most = most && walk.next(p, ny);
    }
  }
  tc_fence_before();
  named_bar_sync(1, NUM_THREADS);
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace weigh
}  // namespace fa
