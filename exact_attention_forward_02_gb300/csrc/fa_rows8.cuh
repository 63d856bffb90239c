// fa_rows8.cuh -- attention of few rows (single tokens, drafts: up to 16 rows of a key head) over a paged cache
// held in 8 bits. Included by fa_rows8.cu. Schedule, items and partial states are those of fa_paged.cuh.
//
// Bound by HBM, as long as nothing else takes longer than the loads, which bring a tile of 128 keys and values
// (d = 128: 32 KB) in 1400 cycles to each SM. So the products are transposed and nothing is converted on the
// way from memory to the tensor cores:
//   S^T = K Q^T     [keys x rows]: a K tile as it is held is the left operand, 128 keys = TMEM lanes, and the
//                   rows are split into sums of E4M3 numbers (split_row), side by side as columns: N = 16 for 8
//                   rows of bf16
//   O^T = V^T P^T   [d x rows]: a V tile as it is held is the left operand too (its keys along K), and P^T is
//                   split into four E5M2 numbers side by side, N = 4 R columns: P' = p1 + p2 + p3 + p4 takes
//                   all 11 bits of P' in fp16; what is cut off is half of E5M2's least number, 2^-17, of P' that
//                   reaches 2^11 in the row's largest weight
// A product then costs by its N instead of 128: shared memory carries 256 (loads) + 128 (S) + 128 (PV) of the
// 1400 cycles. What is left is the issue of the products, about 95 cycles each: with 12 of them to a tile from one
// warp the kernel took 1600 cycles a tile, so there are 8, and a warp for S and one for PV.
//
// Thread = key: 8 softmax warps, a warpgroup for the even and one for the odd key tiles, each with its own m, l
// and O~. A row's running maximum m is the same for all keys of a tile, but needs no maximum over them as long as
// no score passes m + 4 (log2), which one barrier with a vote tells; only then is it found (redux, shared memory)
// and O~ rescaled. P' = P v_scale / vref 2^11 <= 2^15, vref as in fa_paged.cuh.
// l stays spread over the threads until the item ends.
//
// The code that an item needs is kept small (wait_compact, loops that are not unrolled): with 16 warps in eight roles
// it passes the instruction cache, and what was fetched again for each item cost 5 us an item (64 ragged sequences:
// 125 us with two key tiles a step and unrolled ends, 94 without: 5.6 TB/s, 83 % of a copy).
//
// 16 warps: 0-7 softmax, 8 loads K and 11 V, 9 issues S and 12 PV, 10 walks the items, 13 splits queries, up to two
// items ahead, 14 and 15 join the two warpgroups' states and write them out, while those go on with the next item.
#pragma once

#include "fa_paged.cuh"

namespace fa {
namespace paged {

constexpr int R8_THREADS = 512, R8_WARP_PV = 12, R8_WARP_SPLIT = 13, R8_WARP_JOIN = 14;
constexpr float R8_THRESHOLD = 4.0f;  // log2 units

struct Barriers8 : Barriers {
  uint64_t vt_full[MAX_SLOTS], vt_release[MAX_SLOTS];
  uint64_t q2_full[2], q2_empty[2];
  uint64_t st_full[2][2], pt_full[2][2];  // [warpgroup][buffer]
  uint64_t pv_done[2];
  uint64_t vote[2];
  uint64_t join_full[2], join_empty[2];  // [item & 1]
  alignas(16) int said[2][2][4];  // [warpgroup][round & 1][warp]
};

template <int D, int TERMS, int R>
struct Layout8 {
  static constexpr int NQ = (TERMS * R + 15) / 16 * 16, NP = 4 * R;  // columns of S^T and of O^T
  static constexpr int TILE_BYTES = BM * D;
  static constexpr int Q_BYTES = NQ * D;    // row: term R + row
  static constexpr int P_BYTES = BN * NP;  // a row of NP bytes for each key
  // what the warpgroups leave for the joining warps, of JOINS items: O~ [2][R][D], m [2][R], l [2][4][R], units [2]
  static constexpr int JOINS = 2, STATE_FLOATS = 10 * R + 4;
  static constexpr int STAGE_BYTES = JOINS * 2 * R * D * 4;
  // ... and a vote's maxima [2][4][R]; exponents of eight items' rows
  static constexpr int STATE_BYTES = (JOINS * STATE_FLOATS + 8 * R) * 4, EXP_BYTES = 8 * 32;
  static constexpr int HEAD_BYTES = 1280;
  static constexpr int REST = SMEM_LIMIT - 2 * Q_BYTES - 2 * P_BYTES - STAGE_BYTES - STATE_BYTES - EXP_BYTES - HEAD_BYTES - 1024;
  static constexpr int FIT = REST / (2 * TILE_BYTES);
  static constexpr int SLOTS = FIT > MAX_SLOTS ? MAX_SLOTS : FIT;  // of K tiles, and of V tiles
  static constexpr int OFF_K = 0, OFF_V = SLOTS * TILE_BYTES, OFF_P = 2 * SLOTS * TILE_BYTES;
  static constexpr int OFF_Q = OFF_P + 2 * P_BYTES, OFF_STAGE = OFF_Q + (2 * Q_BYTES + 1023) / 1024 * 1024;
  static constexpr int OFF_STATE = OFF_STAGE + STAGE_BYTES, OFF_EXP = OFF_STATE + STATE_BYTES;
  static constexpr int OFF_BAR = OFF_EXP + EXP_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + HEAD_BYTES;
  static constexpr uint32_t TMEM_S = 0, TMEM_O = 4 * NQ;  // S^T of both warpgroups, two tiles each, then O^T of both
  static_assert(sizeof(Barriers8) <= HEAD_BYTES && SLOTS >= 3 && SMEM_BYTES <= SMEM_LIMIT,
                "shared memory budget");
  static_assert(R % 8 == 0 && R <= 16 && 4 * NQ + 2 * NP <= 512, "Tensor Memory");
};

template <int R>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[R]) {
  if constexpr (R == 8) tmem_ld8(taddr, r);
  else tmem_ld16(taddr, r);
}
template <int R>
__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const uint32_t (&r)[R]) {
  if constexpr (R == 8) tmem_st8(taddr, r);
  else tmem_st16(taddr, r);
}

// Sums over the warp's lanes of R values each: the sum of v[r] in lane r (of every R lanes).
template <int R>
__device__ __forceinline__ float lane_sums(float (&v)[R], int lane) {
#pragma unroll
  for (int n = R / 2; n; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], have = up ? v[i + n] : v[i];
      v[i] = have + __shfl_xor_sync(0xffffffffu, give, n);
    }
  }
  float s = v[0];
#pragma unroll
  for (int n = R; n < 32; n <<= 1) s += __shfl_xor_sync(0xffffffffu, s, n);
  return s;
}

template <int D, bool BF16, int R>
__global__ void __launch_bounds__(R8_THREADS, 1)
    fa_paged_rows8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ Params p) {
  constexpr int TERMS = BF16 ? 2 : 3, ROWS = 32;  // rows of a partial state
  using LY = Layout8<D, TERMS, R>;
  constexpr int ITEM_UNITS = 2, SLOTS = LY::SLOTS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, FA_ERR_ALIGN);
    return;
  }
  Barriers8* bars = reinterpret_cast<Barriers8*>(smem + LY::OFF_BAR);
  const uint32_t sK = smem_u32(smem + LY::OFF_K), sV = smem_u32(smem + LY::OFF_V), sP = smem_u32(smem + LY::OFF_P);
  const uint32_t sQ = smem_u32(smem + LY::OFF_Q);
  signed char* exps = reinterpret_cast<signed char*>(smem + LY::OFF_EXP);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(smem_u32(&bars->kv_full[s]), 1);
      mbar_init(smem_u32(&bars->kv_release[s]), 1);
      mbar_init(smem_u32(&bars->vt_full[s]), 1);
      mbar_init(smem_u32(&bars->vt_release[s]), 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_u32(&bars->q2_full[g]), 1);
      mbar_init(smem_u32(&bars->q2_empty[g]), 1);
      for (int x = 0; x < 2; ++x) {
        mbar_init(smem_u32(&bars->st_full[g][x]), 1);
        mbar_init(smem_u32(&bars->pt_full[g][x]), 4);
      }
      mbar_init(smem_u32(&bars->pv_done[g]), 1);
      mbar_init(smem_u32(&bars->vote[g]), 4);
      mbar_init(smem_u32(&bars->join_full[g]), 8);
      mbar_init(smem_u32(&bars->join_empty[g]), 2);
    }
    mbar_init(smem_u32(&bars->mma_drain), 2);
    for (int s = 0; s < ITEM_SLOTS; ++s) {
      mbar_init(smem_u32(&bars->item_full[s]), 1);
      mbar_init(smem_u32(&bars->item_empty[s]), item_readers(true));
    }
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == WARP_LOAD && lane == 0) {
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
  if (p.direct) {
    __syncthreads();
  } else {
    const int per_thread = (p.B + R8_THREADS - 1) / R8_THREADS;
    const int b0 = min((int)threadIdx.x * per_thread, p.B), b1 = min(b0 + per_thread, p.B);
    Seq seq = {};
    const long long my_units = units_of<1, ITEM_UNITS>(p, b0, b1, seq, blockIdx.x == 0);
    range = plan<1, ITEM_UNITS, MIN_UNITS, R8_THREADS / 32>(p, bars, b0, b1, my_units, seq);
  }
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  uint32_t n_item = 0;
  auto item_next = [&]() -> const Item* {
    const uint32_t s = n_item % ITEM_SLOTS;
    const bool w = wait_compact(smem_u32(&bars->item_full[s]), (n_item / ITEM_SLOTS) & 1u, abort_flag, p, ITEM_WAITS);
    return __all_sync(0xffffffffu, w) ? &bars->items[s] : nullptr;
  };
  auto item_done = [&]() {  // this warp needs nothing more of the item
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[n_item % ITEM_SLOTS]));
    ++n_item;
  };
  auto wait_all = [&](uint64_t* bar, uint32_t par) -> bool {
    return __all_sync(0xffffffffu, wait_compact(smem_u32(bar), par, abort_flag, p));
  };

  if (warp >= WARP_LOAD) {
    regs_dec<regs_other(true)>();
    if (warp == WARP_LOAD || warp == WARP_LOAD2) {
      // ======================================================================= loads
      // A warp for K and one for V, tile by tile, page boxes side by side; tile t of the block goes to slot t mod
      // SLOTS. K is used up to four steps before V, so that the two must not wait for one another.
      const bool is_v = warp == WARP_LOAD2;
      uint64_t* const full = is_v ? bars->vt_full : bars->kv_full;
      uint64_t* const release = is_v ? bars->vt_release : bars->kv_release;
      const uint32_t sTo = is_v ? sV : sK;
      // (Divisions by what the host gives cost a tile 500 of these warps' cycles: shifts and steps instead.)
      const int box_shift = 31 - __clz(p.box_keys), boxes = BN >> box_shift;
      const int tiles_per_page = p.page_size > BN ? p.page_size / BN : 1;
      const int my_box = lane & (boxes - 1);
      const uint32_t box_bytes = (uint32_t)p.box_keys * D, box_off = (uint32_t)my_box * box_bytes;
      const bool issues = lane < boxes;
      uint32_t t = 0, slot = 0, par = 0, mask = 0, last_par = 0;  // t: tiles so far
      bool ok = true;
      auto ask = [&](int b, int window) -> int {  // 32 table entries, one per lane
        const int e = window * 32 + lane;
        return e < p.table_stride ? p.table[(size_t)b * p.table_stride + e] : -1;
      };
      auto check = [&](int page, int len, int window) -> int {  // -1: holds no key; num_pages (zeros): a bad page
        if ((long long)(window * 32 + lane) * p.page_size >= len) return -1;
        if (page >= 0 && page < p.num_pages) return page;
        atomicCAS(p.status, 0, FA_ERR_RANGE);
        return p.num_pages;
      };
      auto entry_of = [&](int j) { return p.page_size > BN ? j / tiles_per_page : j * boxes; };  // a tile's first
      int early_b = -1, early_window = 0, early = 0;  // of the block's first tile, before its item has come
      if (p.direct) {
        if (p.whole) early_b = (int)blockIdx.x / p.direct / p.Hkv;
      } else if (range.u0 < range.u1) {
        early_b = bars->start.b;
        early_window = entry_of((int)max(bars->start.off - (long long)ITEM_UNITS, 0ll)) >> 5;
      }
      if (early_b >= 0) early = ask(early_b, early_window);
      while (ok) {
        const Item* src = item_next();
        if (!(ok = src != nullptr)) break;
        const Item it = *src;
        item_done();
        if (it.n == 0) break;
        // the next 32 entries are always on their way, and looked at when they are wanted
        int e0 = entry_of(it.j0), inside = p.page_size > BN ? it.j0 - e0 * tiles_per_page : 0, window = e0 >> 5;
        int held = it.b == early_b && window == early_window ? early : ask(it.b, window);
        int next = ask(it.b, window + 1);
        held = check(held, it.len, window);
        early_b = -1;
        for (int i = 0; i < it.n; ++i, ++t) {
          if (e0 >> 5 != window) {
            held = check(e0 >> 5 == window + 1 ? next : ask(it.b, e0 >> 5), it.len, e0 >> 5);
            window = e0 >> 5;
            next = ask(it.b, window + 1);
          }
          const int page = __shfl_sync(0xffffffffu, held, (e0 + my_box) & 31);
          const int keys = it.len - (it.j0 + i) * BN;
          const int live = keys <= 0 ? 0 : min(boxes, (keys + p.box_keys - 1) >> box_shift);
          if (t >= (uint32_t)SLOTS && !(ok = wait_all(&release[slot], par ^ 1u))) break;
          const uint32_t bar = smem_u32(&full[slot]);
          if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)live * box_bytes);
          __syncwarp();
          in_bounds(p, my_box >= live || !issues || (it.h < p.Hkv && page >= 0 && page <= p.num_pages));
          if (issues && my_box < live)
            tma_load_4d(sTo + slot * LY::TILE_BYTES + box_off, is_v ? &tmV : &tmK, bar, 0, inside * BN, it.h, page);
          mask |= 1u << slot;
          last_par = (last_par & ~(1u << slot)) | (par << slot);
          if (++slot == SLOTS) slot = 0, par ^= 1u;
          if (p.page_size <= BN) e0 += boxes;
          else if (++inside == tiles_per_page) inside = 0, ++e0;
        }
      }
      if (!ok && lane == 0)  // every issued copy must land before the block may exit
        for (int s = 0; s < SLOTS; ++s)
          if (mask & (1u << s)) wait_drain(smem_u32(&full[s]), (last_par >> s) & 1u, p);
      __syncwarp();
    } else if (warp == WARP_MMA) {
      // ======================================================================= S^T = K Q^T
      constexpr uint64_t SW = D == 64 ? UMMA_SWIZZLE_64B : UMMA_SWIZZLE_128B;
      constexpr uint32_t SBO = D == 64 ? 512 : 1024;  // 8 rows
      constexpr uint32_t ID_S = umma_idesc_f16(0, 0, 0, BM, LY::NQ);
      const uint64_t dK = umma_smem_desc<SW>(sK, 16, SBO), dQ = umma_smem_desc<SW>(sQ, 16, SBO);
      uint32_t slot = 0, par = 0, s_n[2] = {0, 0};  // K's ring; tiles of the warpgroups
      bool ok = true;
      while (ok) {
        const Item* src = item_next();
        if (!(ok = src != nullptr)) break;
        const int n = src->n;
        const uint32_t qb = n_item & 1u, q_par = (n_item >> 1) & 1u;
        item_done();
        if (n == 0) break;
        ok = wait_all(&bars->q2_full[qb], q_par);
        const uint64_t b = dQ + ((qb * LY::Q_BYTES) >> 4);
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t g = i & 1, k = s_n[g]++, buf = k & 1u;
          // the buffer is free once the weights of the warpgroup's last tile but one have come (of this item or one
          // before it)
          if (k >= 2 && !(ok = wait_all(&bars->pt_full[g][buf], ((k - 2) >> 1) & 1u))) break;
          if (!(ok = wait_all(&bars->kv_full[slot], par))) break;
          tc_fence_after();
          const uint64_t a = dK + ((slot * LY::TILE_BYTES) >> 4);
          const uint32_t to = tmem + LY::TMEM_S + (2 * g + buf) * LY::NQ;
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < D / 32; ++x) umma_ss_f8(to, a + (x * 32 >> 4), b + (x * 32 >> 4), ID_S, x > 0 ? 1u : 0u);
            umma_commit(smem_u32(&bars->kv_release[slot]));
            umma_commit(smem_u32(&bars->st_full[g][buf]));
            if (i == n - 1) umma_commit(smem_u32(&bars->q2_empty[qb]));
          }
          __syncwarp();
          if (++slot == SLOTS) slot = 0, par ^= 1u;
        }
      }
      if (elect_one()) umma_commit(smem_u32(&bars->mma_drain));
      __syncwarp();
      wait_drain(smem_u32(&bars->mma_drain), 0, p);
      __syncwarp();
    } else if (warp == R8_WARP_PV) {
      // ======================================================================= O^T = V^T P^T
      // both operands along their columns (A: d, B: rows of q), A E4M3, B E5M2. d = 64: lanes 64.. of O^T repeat
      // the others (the offset from one span of 64 columns to the next is 0)
      constexpr uint64_t SW = D == 64 ? UMMA_SWIZZLE_64B : UMMA_SWIZZLE_128B;
      constexpr uint64_t SW_P = R == 8 ? UMMA_SWIZZLE_32B : UMMA_SWIZZLE_64B;
      constexpr uint32_t ID_O = umma_idesc_f16(0, 1, 1, BM, LY::NP) | (1u << 10);
      const uint64_t dV = umma_smem_desc<SW>(sV, 0, D == 64 ? 512 : 1024), dP = umma_smem_desc<SW_P>(sP, 0, 8 * LY::NP);
      uint32_t slot = 0, par = 0, p_n[2] = {0, 0};
      bool ok = true;
      while (ok) {
        const Item* src = item_next();
        if (!(ok = src != nullptr)) break;
        const int n = src->n, j0 = src->j0, len = src->len;
        item_done();
        if (n == 0) break;
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t g = i & 1, k = p_n[g]++;
          if (!(ok = wait_all(&bars->vt_full[slot], par))) break;
          const long long keys = len - (long long)(j0 + i) * BN;
          if (keys < BN) {  // what lies behind the last key may be NaN, which P's zeros do not silence
            const int from = keys < 0 ? 0 : (int)keys * D;
#pragma unroll 1
            for (int x = from + lane * 16; x < LY::TILE_BYTES; x += 512)
              st_shared_v4(sV + slot * LY::TILE_BYTES + x, 0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (!(ok = wait_all(&bars->pt_full[g][k & 1u], (k >> 1) & 1u))) break;
          tc_fence_after();
          const uint64_t a = dV + ((slot * LY::TILE_BYTES) >> 4), b = dP + ((g * LY::P_BYTES) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < BN / 32; ++x)
              umma_ss_f8(tmem + LY::TMEM_O + g * LY::NP, a + (x * 32 * D >> 4), b + (x * 32 * LY::NP >> 4), ID_O,
                         i >= 2 || x > 0 ? 1u : 0u);
            umma_commit(smem_u32(&bars->vt_release[slot]));
            umma_commit(smem_u32(&bars->pv_done[g]));  // O~ is up to date, and P has been read
          }
          __syncwarp();
          if (++slot == SLOTS) slot = 0, par ^= 1u;
        }
      }
      if (elect_one()) umma_commit(smem_u32(&bars->mma_drain));
      __syncwarp();
      wait_drain(smem_u32(&bars->mma_drain), 0, p);
      __syncwarp();
    } else if (warp == R8_WARP_SPLIT) {
      // ======================================================================= queries
      constexpr int QL = D / 8, Q_TURN = 32 / QL;  // lanes of a row, rows at a time
      const int ct = lane, ql = ct % QL;
      bool ok = true;
      while (ok) {
        const Item* src = item_next();
        if (!(ok = src != nullptr)) break;
        const Item it = *src;
        const uint32_t n = n_item;
        item_done();
        if (it.n == 0) break;
        const int rows = it.nt * p.G;
        in_bounds(p, it.tok0 >= 0 && it.tok0 + it.nt <= p.T && (it.h + 1) * p.G <= p.q.H);
        auto load = [&](int r) {  // (zeros where there is no row)
          if (r >= rows) return make_uint4(0, 0, 0, 0);
          const int tok = token_of_row(p, r);
          return *reinterpret_cast<const uint4*>(p.q.ptr + (long long)(it.tok0 + tok) * p.q.ts +
                                                 (long long)(it.h * p.G + r - tok * p.G) * p.q.hs + ql * 8);
        };
        uint4 u = load(ct / QL);
        ok = wait_all(&bars->q2_empty[n & 1u], ((n >> 1) & 1u) ^ 1u);
        if (!ok) break;
#pragma unroll 1
        for (int r = ct / QL; r < R; r += Q_TURN) {
          const uint4 next = load(r + Q_TURN);
          uint32_t w[TERMS][2];
          const int ex = split_row<D, BF16>(u, w);
          u = next;
          // Item n + 8's come when S of item n + 6 has been issued, so the weights of n + 4 have come from the first
          // warpgroup, and the states of n + 1 from both (join_empty).
          if (ql == 0) exps[(n & 7u) * 32 + r] = (signed char)ex;
          const uint32_t sw = D == 128 ? r & 7u : (r >> 1) & 3u;  // R is a multiple of 8: the same for every term
#pragma unroll
          for (int m = 0; m < TERMS; ++m)
            st_shared_v2(sQ + (n & 1u) * LY::Q_BYTES + (m * R + r) * D + ((((uint32_t)ql >> 1) ^ sw) << 4) + (ql & 1) * 8,
                         w[m][0], w[m][1]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->q2_full[n & 1u]));
      }
    } else if (warp >= R8_WARP_JOIN) {
      // ======================================================================= join
      // A row's two states become one (lane = row), then thread = 4 columns of a row.
      const int jt = (int)threadIdx.x - R8_WARP_JOIN * 32;
      bool ok = true;
      while (ok) {
        const Item* src = item_next();
        if (!(ok = src != nullptr)) break;
        const Item it = *src;
        const uint32_t n = n_item, at = n % LY::JOINS;
        item_done();
        if (it.n == 0) break;
        ok = __all_sync(0xffffffffu, wait_compact(smem_u32(&bars->join_full[at]), (n / LY::JOINS) & 1u, abort_flag, p, ITEM_WAITS));
        if (!ok) break;
        const float* st = reinterpret_cast<const float*>(smem + LY::OFF_STATE) + at * LY::STATE_FLOATS;
        const float* stage = reinterpret_cast<const float*>(smem + LY::OFF_STAGE) + at * (2 * R * D);
        const bool partial = it.n != it.ntot;
        const int rows = it.nt * p.G;
        float* part = p.parts + (size_t)(blockIdx.x * 2 + it.slot) * part_floats(D, ROWS);
        auto storable = [&](int token, int head) {
          return in_bounds(p, it.tok0 >= 0 && it.tok0 + token < p.T && it.h * p.G + head < p.o.H &&
                                  (!partial || (blockIdx.x * 2 + it.slot + 1ll) * part_floats(D, ROWS) <= p.parts_len));
        };
        float f[2];
        {
          const int r = lane < R ? lane : 0;
          const int tok = token_of_row(p, r), head = r - tok * p.G;
          const bool sees = (p.causal ? min(it.vis0 + tok, it.len) : it.len) > 0;
          float l[2], m[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float* q = st + 2 * R + 4 * y * R + r;
            l[y] = (q[0] + q[R]) + (q[2 * R] + q[3 * R]);
            // a warpgroup that has seen no key for the row has a sum of exactly 0, and no maximum
            m[y] = l[y] == 0.f ? -INFINITY : st[y * R + r];
          }
          const float mm = fmaxf(m[0], m[1]);
          float sum = 0.f;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            f[y] = m[y] == -INFINITY ? 0.f : ex2_approx(m[y] - mm);
            sum += l[y] * f[y];
            f[y] *= st[10 * R + y] * (1.f / 2048.f);  // O~'s unit
          }
          if (!partial) {
            const float inv = sees ? 1.f / sum : 0.f;
            f[0] *= inv;
            f[1] *= inv;
          }
          if (jt < rows && storable(tok, head)) {  // (at most 32 rows: the first of the two warps)
            if (partial) *reinterpret_cast<float2*>(part + ROWS * D + 2 * r) = make_float2(sees ? mm : -INFINITY, sum);
            else if (p.L) p.L[(long long)(it.tok0 + tok) * (p.Hkv * p.G) + it.h * p.G + head] = sees ? (mm + log2f(sum)) * 0.69314718055994531f : -INFINITY;
          }
        }
        const bool both = it.n > 1;
#pragma unroll 2
        for (int x = jt; x < (rows * (D / 4) + 31) / 32 * 32; x += 64) {
          const int r = x / (D / 4), col = x % (D / 4) * 4;
          const float f0 = __shfl_sync(0xffffffffu, f[0], r), f1 = __shfl_sync(0xffffffffu, f[1], r);
          const int tok = token_of_row(p, r), head = r - tok * p.G;
          if (r >= rows || !storable(tok, head)) continue;
          float4 a = *reinterpret_cast<const float4*>(stage + r * D + col);
          a.x *= f0, a.y *= f0, a.z *= f0, a.w *= f0;
          if (both) {
            const float4 e = *reinterpret_cast<const float4*>(stage + (R + r) * D + col);
            a.x = fmaf(e.x, f1, a.x), a.y = fmaf(e.y, f1, a.y), a.z = fmaf(e.z, f1, a.z), a.w = fmaf(e.w, f1, a.w);
          }
          if (partial) {
            *reinterpret_cast<float4*>(part + (size_t)r * D + col) = a;
          } else {
            uint16_t* dst = p.o.ptr + (long long)(it.tok0 + tok) * p.o.ts + (long long)(it.h * p.G + head) * p.o.hs + col;
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(a.x, a.y), pack2<BF16>(a.z, a.w));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->join_empty[at]));
      }
    } else if (warp == WARP_WALK) {
      if (lane == 0) publish_items<1, ITEM_UNITS, true>(p, bars, range, abort_flag);
      __syncwarp();
    }
    tc_fence_before();
    named_bar_sync(1, R8_THREADS);
    if (warp == WARP_MMA) {
      tc_fence_after();
      tmem_dealloc(tmem, TMEM_COLS);
    }
  } else {
    regs_inc<regs_softmax(true)>();
    // ======================================================================= softmax
    const int g = warp >> 2, wq = warp & 3, kk = wq * 32 + lane;  // the thread's key in a tile, its lane of TMEM
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + LY::TMEM_S + 2 * g * LY::NQ, tO = tmem + lane_off + LY::TMEM_O + g * LY::NP;
    const uint32_t myP = sP + (uint32_t)(g * LY::P_BYTES + kk * LY::NP);
    const uint32_t sw = R == 8 ? (kk >> 2) & 1 : (kk >> 1) & 3;  // swizzle of the row's pieces
    float* const tops = reinterpret_cast<float*>(smem + LY::OFF_STATE) + LY::JOINS * LY::STATE_FLOATS + g * 4 * R;  // [4][R]
    // Tiles of the warpgroup so far. Its products P V are waited for one by one, before the next one's weights are
    // given out, so that their barrier is never a phase ahead (which its parity could not tell).
    uint32_t kt = 0;
    bool ok = true;
    auto wait_pv = [&]() {
      if (kt) ok = ok && wait_all(&bars->pv_done[g], (kt - 1) & 1u);
    };
    // Whether all threads of the warpgroup say so; a barrier for them as well, and bounded like every wait (a warp
    // that gave up clears ok).
    uint32_t v_n = 0;
    auto vote = [&](bool all) -> bool {
      all = __all_sync(0xffffffffu, all);
      int* said = bars->said[g][v_n & 1u];
      if (lane == 0) {
        said[wq] = all;
        mbar_arrive(smem_u32(&bars->vote[g]));
      }
      ok = ok && wait_all(&bars->vote[g], v_n & 1u);
      ++v_n;
      uint32_t x[4];
      ld_shared_u4(smem_u32(said), x);
      return ok && x[0] && x[1] && x[2] && x[3];
    };
    while (ok) {
      const Item* item = item_next();
      if (!(ok = item != nullptr) || item->n == 0) break;
      const int n = item->n, rows = item->nt * p.G, vis0 = item->vis0, len = item->len;
      // keys that the first row sees; with a causal mask row r sees token_of_row(r) more
      const int sees0 = p.causal ? min(vis0, len) : len;
      uint64_t c2[R / 2], nm2[R / 2], l2[R / 2];  // c 2^e, -m and l of pairs of rows
      float vref = 1.f, vinv = 2048.f;
#pragma unroll
      for (int r = 0; r < R / 2; ++r) nm2[r] = l2[r] = 0, c2[r] = 0;
      // Lane x < 16 has the scales of key group x (8 keys) of a tile. The next tile's, and the page of the one after
      // that, are on their way.
      const int j0 = item->j0, h = item->h;
      const int* table = p.table + (size_t)item->b * p.table_stride;
      auto ask_page = [&](int i) -> int {
        const int key = (j0 + i) * BN + lane * 8;  // (below 2^31: the table covers at most 0x7fffff00 keys)
        if (i >= n || lane >= 16 || key >= len) return -1;
        return table[p.page_shift >= 0 ? (uint32_t)key >> p.page_shift : (uint32_t)key / (uint32_t)p.page_size];
      };
      auto ask_scales = [&](int page, float& ks, float& vs) {  // of no key, and of a bad page (zeros): 1 and 0
        ks = 1.f;
        vs = 0.f;
        if (page < 0 || page >= p.num_pages) return;
        const size_t at = (size_t)page * p.Hkv + h;
        ks = p.ks[at];
        vs = p.vs[at];
      };
      float ks_now, vs_now, ks_next = 1.f, vs_next = 0.f;
      int page_next = -1;
#pragma unroll 1
      for (int i = g - 4; i < n; i += 2) {  // (the first two rounds only ask)
        ks_now = ks_next;
        vs_now = vs_next;
        ask_scales(page_next, ks_next, vs_next);
        page_next = ask_page(i + 4);
        if (i < 0) continue;
        const uint32_t buf = kt & 1u;
        ok = wait_all(&bars->st_full[g][buf], (kt >> 1) & 1u);
        if (!ok) break;
        tc_fence_after();
        if (i < 2) {  // the item's exponents, written before its first product
          const signed char* ex = exps + (n_item & 7u) * 32;
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            const float x = r * 2 < rows ? p.c * __uint_as_float((uint32_t)(127 + ex[2 * r]) << 23) : 0.f;
            const float y = r * 2 + 1 < rows ? p.c * __uint_as_float((uint32_t)(127 + ex[2 * r + 1]) << 23) : 0.f;
            c2[r] = f2(x, y);
          }
        }
        // x = score in log2 units, -inf for what a row does not see; rows that are none stay at 0
        uint64_t x2[R / 2];
        {
          uint32_t sr[TERMS][R];
#pragma unroll
          for (int x = 0; x < TERMS; ++x) tmem_ld_n<R>(tS + buf * LY::NQ + x * R, sr[x]);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < TERMS; ++x) reg_fence(sr[x]);
          const float ks = __shfl_sync(0xffffffffu, ks_now, kk >> 3);
          const uint64_t ks2 = f2(ks, ks);
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            auto pair = [&](int x) { return f2(__uint_as_float(sr[x][2 * r]), __uint_as_float(sr[x][2 * r + 1])); };
            uint64_t sum = pair(TERMS - 1);  // small ones first
#pragma unroll
            for (int x = TERMS - 2; x >= 0; --x) sum = f2_add(sum, pair(x));
            x2[r] = f2_mul(f2_mul(sum, ks2), c2[r]);
          }
        }
        if ((j0 + i + 1) * BN > sees0) {
          const int key = (j0 + i) * BN + kk;
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            float a, e;
            f2_split(x2[r], a, e);
            auto sees = [&](int row) { return key < (p.causal ? min(vis0 + token_of_row(p, row), len) : len); };
            if (2 * r < rows && !sees(2 * r)) a = -INFINITY;
            if (2 * r + 1 < rows && !sees(2 * r + 1)) e = -INFINITY;
            x2[r] = f2(a, e);
          }
        }
        wait_pv();  // O~ is up to date, and the buffer of P has been read
        if (!ok) break;
        // the largest scale of V (positive numbers in the order of their bits), the same in all warps
        const float vt = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vs_now)));
        const bool same_unit = vt <= vref;
        float most = INFINITY;
        if (i >= 2) {
          most = -INFINITY;
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            float a, e;
            f2_split(f2_add(x2[r], nm2[r]), a, e);
            most = max3(most, a, e);
          }
        }
        if (!vote(most <= R8_THRESHOLD && same_unit)) {
          if (!ok) break;
          // New maxima of the rows that have passed the threshold (all of them in the item's first tile), and a
          // new unit of V where a larger scale has come. (Before the tops are written again there is another vote.)
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            float a, e;
            f2_split(x2[r], a, e);
            a = warp_max(a);
            e = warp_max(e);
            if (lane == 0) *reinterpret_cast<float2*>(tops + wq * R + 2 * r) = make_float2(a, e);
          }
          vote(true);
          if (!ok) break;
          float beta = 1.f;
          if (i < 2 || !same_unit) {
            const float v_new = fmaxf(vt, 7.8886090522101181e-31f);  // 2^-100: pages of zeros
            beta = __fdividef(vref, v_new);
            vref = v_new;
            vinv = __fdividef(2048.f, v_new);
          }
          uint64_t al2[R / 2];
#pragma unroll
          for (int r = 0; r < R / 2; ++r) {
            float m[2], nm[2], al[2];
            f2_split(nm2[r], nm[0], nm[1]);
            const float2 t0 = *reinterpret_cast<const float2*>(tops + 2 * r), t1 = *reinterpret_cast<const float2*>(tops + R + 2 * r);
            const float2 t2 = *reinterpret_cast<const float2*>(tops + 2 * R + 2 * r), t3 = *reinterpret_cast<const float2*>(tops + 3 * R + 2 * r);
            m[0] = fmaxf(fmaxf(t0.x, t1.x), fmaxf(t2.x, t3.x));
            m[1] = fmaxf(fmaxf(t0.y, t1.y), fmaxf(t2.y, t3.y));
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              al[y] = 1.f;
              if (2 * r + y < rows && m[y] != -INFINITY && (i < 2 || m[y] + nm[y] > R8_THRESHOLD)) {
                if (i >= 2) al[y] = ex2_approx(-m[y] - nm[y]);
                nm[y] = -m[y];
              }
            }
            nm2[r] = f2(nm[0], nm[1]);
            al2[r] = f2(al[0], al[1]);
            l2[r] = f2_mul(l2[r], al2[r]);
          }
          if (i >= 2) {
            tc_fence_after();
            const uint64_t be2 = f2(beta, beta);
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {  // terms of P
              uint32_t o[R];
              tmem_ld_n<R>(tO + x * R, o);
              tmem_wait_ld();
              reg_fence(o);
#pragma unroll
              for (int r = 0; r < R / 2; ++r) {
                float a, e;
                f2_split(f2_mul(f2(__uint_as_float(o[2 * r]), __uint_as_float(o[2 * r + 1])), f2_mul(al2[r], be2)), a, e);
                o[2 * r] = __float_as_uint(a);
                o[2 * r + 1] = __float_as_uint(e);
              }
              tmem_st_n<R>(tO + x * R, o);
            }
            tmem_wait_st();
          }
        }
        // P' in fp16, as four E5M2 terms: byte (term R + row) of the key's row
        const float fv = __shfl_sync(0xffffffffu, vs_now, kk >> 3) * vinv;
        const uint64_t fv2 = f2(fv, fv);
        uint32_t term[4][R / 4];
#pragma unroll
        for (int r = 0; r < R / 2; r += 2) {
          uint32_t hh[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            float a, e;
            f2_split(f2_add(x2[r + z], nm2[r + z]), a, e);
            const uint64_t pr = f2(ex2_approx(a), ex2_approx(e));
            l2[r + z] = f2_add(l2[r + z], pr);
            f2_split(f2_mul(pr, fv2), a, e);
            hh[z] = pack2<false>(a, e);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t b0 = pack2_e5m2(hh[0]), b1 = pack2_e5m2(hh[1]);
            term[x][r / 2] = __byte_perm(b0, b1, 0x5410);
            if (x < 3) {
              hh[0] = sub_f16x2(hh[0], unpack2_e5m2(b0));
              hh[1] = sub_f16x2(hh[1], unpack2_e5m2(b1));
            }
          }
        }
        const uint32_t* flat = &term[0][0];
#pragma unroll
        for (uint32_t j = 0; j < R / 4; ++j)  // 16-byte pieces
          st_shared_v4(myP + ((j ^ sw) << 4), flat[4 * j], flat[4 * j + 1], flat[4 * j + 2], flat[4 * j + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->pt_full[g][buf]));
        ++kt;
      }
      if (!ok) break;
      // ------------------------------------------------------------------ the state, for the joining warps
      const bool worked = n > g;
      const uint32_t at = n_item % LY::JOINS, round = n_item / LY::JOINS;
      float l[R];
#pragma unroll
      for (int r = 0; r < R / 2; ++r) f2_split(l2[r], l[2 * r], l[2 * r + 1]);
      const float sum = lane_sums<R>(l, lane);
      if (round > 0) ok = wait_all(&bars->join_empty[at], (round - 1) & 1u);
      wait_pv();
      if (!ok) break;
      float* st = reinterpret_cast<float*>(smem + LY::OFF_STATE) + at * LY::STATE_FLOATS;
      if (lane < R) st[2 * R + (g * 4 + wq) * R + lane] = sum;
      if (wq == 0 && lane == 0) {
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
          float a, e;
          f2_split(nm2[r], a, e);
          *reinterpret_cast<float2*>(st + g * R + 2 * r) = make_float2(-a, -e);
        }
        st[10 * R + g] = vref;
      }
      if (worked) {
        tc_fence_after();
        float o_sum[R] = {};
#pragma unroll 1
        for (int x = 3; x >= 0; --x) {  // terms, small ones first
          uint32_t o[R];
          tmem_ld_n<R>(tO + x * R, o);
          tmem_wait_ld();
          reg_fence(o);
#pragma unroll
          for (int r = 0; r < R; ++r) o_sum[r] += __uint_as_float(o[r]);
        }
        float* stage = reinterpret_cast<float*>(smem + LY::OFF_STAGE) + at * (2 * R * D) + g * (R * D) + kk;
        if (kk < D) {  // lane of TMEM = column of O
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (r < rows) stage[r * D] = o_sum[r];
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->join_full[at]));
      item_done();
    }
    tc_fence_before();
    named_bar_sync(1, R8_THREADS);
  }
}

}  // namespace paged
}  // namespace fa
