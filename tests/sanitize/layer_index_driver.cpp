// Walks the index arithmetic of the paged-cache kernels on the host, as the
// kernels use it, over random batches whose device arrays hold anything: every
// index stays in its array, and every visible key is met exactly once.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "layer_index.h"

using namespace ocq;

static int failed = 0;
#define CHECK(x) do { if (!(x)) { ++failed; std::printf("line %d: %s\n", __LINE__, #x); } } while (0)

int main() {
  std::mt19937 rng(7);
  auto below = [&](int n) { return (int)(rng() % (unsigned)n); };
  for (int trial = 0; trial < 3000; ++trial) {
    const bool garbage = trial % 3 == 0;
    const int requests = 1 + below(4), group = 1 + below(8), shift = below(7), max_pages = 1 + below(40);
    const int num_pages = 1 + below(50), TT = 32 << below(3), rows_tile = 16 << below(4), splits = 1 + below(5);
    const int window = below(3) ? 1 + below(200) : 0, sinks = window ? below(3) * below(100) : 0;
    std::vector<int32_t> q_start(requests + 1), kv_lens(requests), table(max_pages);
    for (int r = 0; r < requests; ++r) q_start[r + 1] = q_start[r] + below(3) * below(30);
    const int tokens = q_start[requests] > 0 ? q_start[requests] : 1;
    for (int& x : kv_lens) x = below((max_pages << shift) + 1);
    if (garbage) {
      for (int& x : q_start) if (below(2)) x = (int)rng();
      for (int& x : kv_lens) if (below(2)) x = (int)rng();
    }
    for (int& x : table) x = below(4) ? below(num_pages) : (int)rng();   // some pages are none
    for (int req = 0; req < requests; ++req) {
      const Span sp = token_span(q_start.data(), req, tokens);
      if (sp.n <= 0) continue;
      CHECK(sp.t0 >= 0 && sp.t0 + sp.n <= tokens);
      const int kv = kv_bound(kv_lens[req], max_pages, shift);
      CHECK(kv >= 0 && kv <= max_pages << shift);
      const int base = kv - sp.n;
      for (int row0 = 0; row0 < sp.n * group; row0 += rows_tile) {
        const int last = (row0 + rows_tile < sp.n * group ? row0 + rows_tile : sp.n * group) - 1;
        const KeyTiles k = key_tiles(base + row0 / group, base + last / group, window, sinks, TT);
        CHECK(k.total >= 0 && k.sink_tiles <= k.lo_tile);
        std::vector<int> met(kv + 2 * TT + 1, 0);
        const int per = (k.total + splits - 1) / splits;
        for (int split = 0; split < splits; ++split) {
          const int s0 = split * per < k.total ? split * per : k.total, s1 = s0 + per < k.total ? s0 + per : k.total;
          for (int t = s0; t < s1; ++t)
            for (int x = 0; x < TT; ++x) {
              const int key = tile_of(k, t) * TT + x;
              CHECK(key >= 0 && key < (int)met.size());
              ++met[key];
              const int e = table_entry(key, kv, shift);
              CHECK(e >= 0 && e < max_pages);
              const KeyRange range = key_range(base + row0 / group, base + last / group, window, sinks);
              bool any = false;
              for (int row = row0; row <= last; row += group) any |= key_seen(key, base + row / group, window, sinks);
              any |= key_seen(key, base + last / group, window, sinks);
              CHECK(key_in(key, range) == any);
              if (key > range.from && key <= range.to) CHECK(any);   // no test needed inside
              if (page_there(table[e], num_pages) && key_in(key, range)) {
                CHECK(key < kv);
                const uint64_t off = row_offset(key, table[e], shift, 1u << (shift + 20), 1u << 20);
                CHECK(off < (uint64_t)num_pages << (shift + 20));
              }
            }
        }
        for (int row = row0; row <= last; ++row) {
          const int place = base + row / group;
          for (int j = 0; j < kv; ++j)
            if (key_seen(j, place, window, sinks)) CHECK(met[j] == 1);
          CHECK(!key_seen(kv, place, window, sinks));
        }
      }
    }
  }
  // pieces: never more than tiles, none empty, and no more than the slots at
  // the bound
  for (int trial = 0; trial < 20000; ++trial) {
    const int requests = 1 + below(64), kv_heads = 1 + below(8), segments = requests * kv_heads;
    const int slots = 2 * segments + below(600);
    std::vector<int> T(requests);
    int total = 0;
    for (int& x : T) {
      x = below(4) ? 1 + below(1 << below(20)) : 0;
      if (x > (1 << 30) / segments) x = (1 << 30) / segments;
      total += x * kv_heads;
    }
    const int bound = piece_bound(total, segments, slots);
    for (int per : {1, 1 + below(50), bound}) {
      long long pieces = 0;
      for (int x : T) {
        const int c = piece_count(x, 1.0f / (float)per);
        CHECK(c >= (x > 0) && c <= x);
        pieces += (long long)c * kv_heads;
        for (int k = 0; c > 0 && k < 20; ++k) {
          const int i = below(c);
          CHECK(piece_begin(x, i + 1, c) > piece_begin(x, i, c) && piece_begin(x, 0, c) == 0 &&
                piece_begin(x, c, c) == x);
        }
      }
      if (per == bound) CHECK(pieces <= slots);
    }
  }
  std::printf("OK (%d failed checks)\n", failed);
  return failed != 0;
}
