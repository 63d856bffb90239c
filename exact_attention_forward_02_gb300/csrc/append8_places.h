// append8_places.h -- where the units of the append to an 8-bit cache belong: plain index arithmetic, of the kernel
// (fa_append8.cuh) and, compiled for the host, of its tests.
//
// A sequence with token rows [c0, c1) reaches at most floor(c1 / page) - floor(c0 / page) + 2 pages, so the places
// floor(c0 / page) + 2 b ... are enough for it, and a place's sequence is found by a search over the offsets.
// Offsets may be anything: where they decrease, the search may end at a sequence whose first place lies behind the
// wanted one, and piece_of turns that down before anything is looked up by it.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define FA_PLACES __host__ __device__ __forceinline__
#else
#define FA_PLACES inline
#endif

namespace fa {

// place of a sequence's first page
FA_PLACES uint32_t first_place(int begin, int page_size, int b) {
  return (uint32_t)(begin > 0 ? begin : 0) / (uint32_t)page_size + 2u * (uint32_t)b;
}

// The last sequence whose first place is at most the wanted one, -1: none. count(lo, step, end): of the sequences
// lo + step - 1, lo + 2 step - 1, ... (32 of them, those before `end`), how many have such a first place.
template <typename F>
FA_PLACES int search_places(int B, F count) {
  int lo = 0, n = B;
  while (n > 0) {
    const int step = (n + 31) / 32, parts = count(lo, step, lo + n);
    lo += parts * step;
    n = step - 1 < n - parts * step ? step - 1 : n - parts * step;
  }
  return (lo < B ? lo : B) - 1;
}

// What place `place` stands for, given the sequence that the search found: its page `at` of the sequence and the slots
// [s0, s1) of it that get new tokens. alive: there are such slots, and 0 <= at page_size < len; nothing else may be used
// where it is false. early: the sequence's first tokens lie before position 0 (said once a sequence).
struct Piece {
  int at, s0, s1;
  bool alive, early;
};
FA_PLACES Piece piece_of(uint32_t place, int b, int begin, int end, int len, int T, int page_size) {
  // (without branches, so that the loads behind the arguments are on their way together; differences of anything, mod 2^32)
  const uint32_t nth = place - first_place(begin, page_size, b);  // page of the sequence's new ones
  const bool rows = begin >= 0 && end > begin && end <= T;
  const int n = (int)((uint32_t)end - (uint32_t)begin), first = len > n ? (int)((uint32_t)len - (uint32_t)n) : 0;
  // 2^30 and more: behind any sequence (pages hold 8 tokens at least), or before this one's first place
  const bool near = nth < 1u << 30;
  const int at = first / page_size + (int)(nth & 0x3fffffffu);
  const long long from = (long long)at * page_size;
  const int left = (int)((uint32_t)len - (uint32_t)from);
  Piece x;
  x.at = at;
  x.s0 = nth == 0 ? (int)((uint32_t)first - (uint32_t)from) : 0;
  x.s1 = left < page_size ? left : page_size;
  x.alive = rows && near && from < len;  // then s0 < s1: first < len, and the page's first slot lies below len too
  x.early = rows && nth == 0 && len < n;
  return x;
}

}  // namespace fa
