// Runs the attention kernel's schedule (csrc/attn_plan.cuh) on the host: every block of every item lies
// in exactly one run, the runs of a split item are those that its merge expects, and sequences of
// billions of units are cut where the cuts say.  Prints what it checked; exits 1 at a mistake.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "attn_plan.cuh"

typedef long long i64;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)

static Seq seq(int n, int kv, int rows) { return Seq{0, n, kv, (n + rows - 1) / rows, false}; }

struct Batch {
  std::vector<Seq> s;
  int rows, heads, causal;
  std::vector<i64> begin;   // first unit of every sequence, and the end
  void count() {
    begin.assign(1, 0);
    for (const Seq& x : s) begin.push_back(begin.back() + tiles_before(x, x.tiles, rows, causal) * heads);
  }
  i64 units() const { return begin.back(); }
};
struct Item { int b, head, t; i64 from; int size, in; };

// the item that holds unit `at`, as the kernel's threads find it together
static Item find(const Batch& B, i64 at) {
  int b = 0;
  while (!(B.begin[b] <= at && at < B.begin[b + 1])) ++b;
  const Seq& s = B.s[b];
  const Spot spot = locate(at - B.begin[b], (B.begin[b + 1] - B.begin[b]) / B.heads);
  CHECK(spot.head >= 0 && spot.head < B.heads);
  int lo = 0, hi = s.tiles;                         // tiles_before grows with the tile
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    (tiles_before(s, mid, B.rows, B.causal) <= spot.unit ? lo : hi) = mid;
  }
  const int size = SETUP + tile_blocks(s, lo, B.rows, B.causal);
  const i64 in = spot.unit - tiles_before(s, lo, B.rows, B.causal);
  CHECK(in >= 0 && in < size);
  return Item{b, spot.head, lo, at - in, size, (int)in};
}

static i64 runs_of(i64 units, int sms) {
  const i64 most = units / MIN_RUN < 1 ? 1 : units / MIN_RUN;
  return most < sms ? most : sms;
}

// every CTA's run of a batch, block by block
static void walk(Batch& B, int sms) {
  B.count();
  const i64 units = B.units(), runs = runs_of(units, sms);
  if (!units) return;
  struct Entry { i64 from; int size; std::vector<int> owner; };
  std::vector<Entry> items;
  for (size_t b = 0; b < B.s.size(); ++b)
    for (int h = 0; h < B.heads; ++h)
      for (int t = 0; t < B.s[b].tiles; ++t) {
        const int blocks = tile_blocks(B.s[b], t, B.rows, B.causal);
        const i64 from = B.begin[b] + h * ((B.begin[b + 1] - B.begin[b]) / B.heads) + tiles_before(B.s[b], t, B.rows, B.causal);
        CHECK(items.empty() ? from == 0 : from == items.back().from + items.back().size);
        items.push_back({from, SETUP + blocks, std::vector<int>(blocks, -1)});
      }
  CHECK(items.back().from + items.back().size == units);
  auto moved = [&](int i) {
    const i64 cut = cut_at(units, runs, i);
    if (cut == units) return units;
    const Item it = find(B, cut);
    return moved_cut(cut, it.in, it.size);
  };
  for (int c = 0; c < runs; ++c) {
    const i64 u0 = moved(c), u1 = moved(c + 1);
    if (u0 >= u1) continue;
    for (Entry& e : items) {
      if (e.from + e.size <= u0 || e.from >= u1) continue;
      const i64 start = e.from + SETUP, blocks = e.size - SETUP;
      const i64 j0 = u0 > start ? u0 - start : 0, j1 = blocks < u1 - start ? blocks : u1 - start;
      CHECK(j0 < j1);
      for (i64 j = j0; j < j1; ++j) { CHECK(e.owner[j] == -1); e.owner[j] = c; }
    }
  }
  for (const Entry& e : items) {
    for (int o : e.owner) CHECK(o >= 0);
    if (e.owner.front() != e.owner.back()) {
      CHECK(first_run(e.from, units, runs) == e.owner.front() && last_run(e.from, e.size, units, runs) == e.owner.back());
      for (size_t j = 1; j < e.owner.size(); ++j) CHECK(e.owner[j] == e.owner[j - 1] || e.owner[j] == e.owner[j - 1] + 1);
    }
  }
}

// cuts of a batch too large to walk
static void cuts(Batch& B, int sms) {
  B.count();
  const i64 units = B.units(), runs = runs_of(units, sms);
  for (int i = 0; i < runs; ++i) {
    const i64 cut = cut_at(units, runs, i);
    CHECK((__int128)cut == (__int128)units * i / runs);
    const Item it = find(B, cut);
    const i64 per = (B.begin[it.b + 1] - B.begin[it.b]) / B.heads;
    CHECK((__int128)B.begin[it.b] + (__int128)it.head * per + tiles_before(B.s[it.b], it.t, B.rows, B.causal) + it.in == cut);
    CHECK(it.from <= cut && cut < it.from + it.size);
    if (cut - it.from > SNAP && it.from + it.size - cut > SNAP) {   // this item is cut here
      const int a = first_run(it.from, units, runs), z = last_run(it.from, it.size, units, runs);
      CHECK(a < i && i <= z);
    }
  }
}

int main() {
  std::mt19937 g(1);
  auto upto = [&](int hi) { return (int)(g() % (unsigned)(hi + 1)); };
  // sums over tiles against direct ones
  for (int k = 0; k < 20000; ++k) {
    const int rows = 1 + upto(255), n = upto(3000), kv = upto(1) ? upto(4000) : n + upto(100000), causal = upto(3) > 0;
    const Seq s = seq(n, kv, rows);
    i64 sum = 0;
    const int stop = s.tiles ? upto(s.tiles) : 0;
    for (int t = 0; t < stop; ++t) sum += SETUP + tile_blocks(s, t, rows, causal);
    CHECK(tiles_before(s, stop, rows, causal) == sum);
  }
  // whole schedules
  for (int k = 0; k < 1500; ++k) {
    Batch B;
    const int kind = upto(3), count = 1 + upto(kind == 0 ? 3 : 40);
    B.rows = 1 + upto(upto(1) ? 255 : 31);
    B.heads = 1 + upto(15);
    B.causal = upto(4) > 0;
    for (int b = 0; b < count; ++b) {
      const int n = kind == 1 ? 1 : kind == 2 ? 1 + upto(15) : upto(600), kv = B.causal && upto(9) == 0 ? upto(n) : n + upto(kind == 3 ? 300 : 6000);
      B.s.push_back(seq(n, kv, B.rows));
    }
    walk(B, 1 + upto(3) * 50 + 1);
  }
  // billions of units: tokens, query heads, key-value heads of prompts on one and two tiles of rows
  const int big[][3] = {{2200000, 64, 8}, {1500000, 128, 8}, {1500000, 128, 128}, {530000, 1024, 16}, {2000000, 1024, 16}, {16000000, 128, 2}, {1000000, 8, 8}};
  i64 most = 0;
  for (const auto& x : big)
    for (int tiles = 1; tiles <= 2; ++tiles) {
      Batch B;
      B.rows = tiles * (BM / (x[1] / x[2]));
      B.heads = x[2];
      B.causal = 1;
      for (int n : {300, x[0], 5000}) B.s.push_back(seq(n, n, B.rows));
      cuts(B, 152);
      most = B.units() > most ? B.units() : most;
    }
  CHECK(most > 1ll << 32);
  std::printf("ok: largest schedule %lld units\n", most);
  return 0;
}
