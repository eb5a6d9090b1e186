// The attention kernel's schedule: items, units, runs and merges (see attn_tile.cuh).
// Whole numbers only, for host and device: counts of units are 64 bits wide
// throughout (a prompt of a million tokens has billions), positions 32.
#pragma once

#ifndef __CUDACC__
#define __host__
#define __device__
#define __forceinline__ inline
#endif

namespace {

constexpr int BN = 128;             // keys per block
constexpr int BM = 128;             // rows per tile (tensor-memory lanes)
// Of the run schedule, in units (about 1.6 us with two tiles, 1.2 with one).  Time over 30 cases of all sizes
// against the values chosen: SETUP and SNAP 2, +2%; SNAP 3, +1%; SNAP 6, +0.4%; SETUP 4, +0.3%; MIN_RUN 2, 5 and
// 8, +1, +7 and +15%.  Without SETUP and SNAP 8 prompts of 100-2048 tokens take 114 instead of 77 us.
constexpr int SETUP = 3;            // units of an item besides its blocks
constexpr int SNAP = 4;             // units that a run gives up or takes on to end with an item (SETUP at least)
constexpr int MIN_RUN = 3;          // units of a CTA at least
constexpr int LEN_MAX = 0x7fffffff - 511;   // tokens of a sequence, cached or packed: positions up to three blocks on fit 32 bits
// sum over i = 0 .. n-1 of floor((a i + b) / m), by the Euclidean reduction that counts the lattice points under a
// line (Graham, Knuth and Patashnik, Concrete Mathematics, section 3.5); a n + b < 2^32
__host__ __device__ inline long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  unsigned long long s = 0;
  while (n > 0) {
    s += (unsigned long long)(n - 1) * n / 2 * (a / m);
    a %= m;
    s += (unsigned long long)n * (b / m);
    b %= m;
    const unsigned y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const unsigned t = m;
    m = a;
    a = t;
  }
  return (long long)s;
}

struct Seq {          // one sequence as the kernel sees it
  int row0, n;        // packed rows
  int kv;             // cached tokens (0 where the length is invalid)
  int tiles;
  bool bad;
};
// key blocks of tile t (at least one, so that its rows are written)
__host__ __device__ __forceinline__ int tile_blocks(const Seq& s, int t, int tile_rows, int causal) {
  const int end = (t + 1) * tile_rows, len = causal ? s.kv - s.n + (end < s.n ? end : s.n) : s.kv;
  const int blocks = (len + BN - 1) / BN;
  return blocks > 1 ? blocks : 1;
}
// units of tiles 0 .. t-1
__host__ __device__ inline long long tiles_before(const Seq& s, int t, int tile_rows, int causal) {
  if (t == 0) return 0;
  if (!causal) return (long long)t * (SETUP + tile_blocks(s, 0, tile_rows, causal));
  long long last = (long long)t * SETUP;
  if (t == s.tiles) {                   // the last tile may be short
    last += tile_blocks(s, t - 1, tile_rows, causal);
    if (--t == 0) return last;
  }
  const int base = s.kv - s.n;          // tile i (from 1) ends at key base + i * tile_rows
  const int below = base >= BN ? 0 : (BN - base) / tile_rows, ones = below < t ? below : t;
  if (ones == t) return last + t;
  return last + ones + floor_sum((unsigned)(t - ones), BN, (unsigned)tile_rows, (unsigned)(base + (ones + 1) * tile_rows + BN - 1));
}

// Where unit `at` of a sequence lies: its units are those of its heads in order, `per_head` each
struct Spot {
  int head;
  long long unit;     // within the head
};
__host__ __device__ inline Spot locate(long long at, long long per_head) {
  const long long head = at / per_head;
  return Spot{(int)head, at - head * per_head};
}

// The cut before run i, of `runs` equal ones; then moved to an item's start or end where one is near, the item
// having `size` units and the cut lying `in` units into it
__host__ __device__ __forceinline__ long long cut_at(long long units, long long runs, int i) { return units * i / runs; }
__host__ __device__ __forceinline__ long long moved_cut(long long cut, int in, int size) {
  return in <= SNAP ? cut - in : size - in <= SNAP ? cut - in + size : cut;
}
// The first and the last run that hold a part of the item of units begin .. begin + size - 1, if it is cut at all
__host__ __device__ __forceinline__ int first_run(long long begin, long long units, long long runs) {
  return (int)(((begin + SNAP + 1) * runs - 1) / units);
}
__host__ __device__ __forceinline__ int last_run(long long begin, int size, long long units, long long runs) {
  return (int)(((begin + size - SNAP) * runs - 1) / units);
}

}  // namespace
