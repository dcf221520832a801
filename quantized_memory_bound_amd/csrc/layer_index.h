// Index arithmetic of the paged-cache kernels, apart from them so that it can
// be checked on the host: every index that comes from a device array is
// bounded here before it is used as an address.
#pragma once
#include <stdint.h>

#ifdef __HIPCC__
#define OCQ_HD __host__ __device__ __forceinline__
#else
#define OCQ_HD inline
#endif

namespace ocq {

// Rows [t0, t0 + n) of the token axis that belong to a request; n <= 0: none.
struct Span {
  int t0, n;
};
OCQ_HD Span token_span(const int32_t* q_start, int req, int tokens) {
  int t0 = q_start[req], t1 = q_start[req + 1];
  t0 = t0 < 0 ? 0 : t0 > tokens ? tokens : t0;
  t1 = t1 < 0 ? 0 : t1 > tokens ? tokens : t1;
  return Span{t0, t1 - t0};
}

// Cached tokens of a request, no more than its row of the page table names.
OCQ_HD int kv_bound(int kv, int max_pages, int page_shift) {
  const int cap = max_pages << page_shift;
  return kv < 0 ? 0 : kv > cap ? cap : kv;
}

// Tiles of TT keys that rows at places p_lo .. p_hi can see: those of the
// first `sinks` tokens, then from the first row's window to the last row's
// place.  Tile t of the `total` starts at key tile_of(t) * TT.
struct KeyTiles {
  int lo_tile, sink_tiles, total;
};
OCQ_HD KeyTiles key_tiles(int p_lo, int p_hi, int window, int sinks, int TT) {
  KeyTiles k{0, 0, 0};
  if (p_hi < 0) return k;
  if (window > 0 && p_lo >= window) {
    const int lo = p_lo - window + 1;
    k.lo_tile = lo / TT;
    const int s = sinks < lo ? sinks : lo;
    k.sink_tiles = s / TT + (s % TT != 0);
    if (k.sink_tiles > k.lo_tile) k.sink_tiles = k.lo_tile;
  }
  k.total = k.sink_tiles + p_hi / TT + 1 - k.lo_tile;
  return k;
}
OCQ_HD int tile_of(const KeyTiles& k, int t) { return t < k.sink_tiles ? t : t - k.sink_tiles + k.lo_tile; }

// Whether key j is visible to a row at `place` (-1: a row that is not there).
OCQ_HD bool key_seen(int j, int place, int window, int sinks) {
  return j <= place && (window <= 0 || j > place - window || j < sinks);
}

// Entry of a request's page-table row that names key's page; keys past the
// last one take the last one's (their rows are not loaded).
OCQ_HD int table_entry(int key, int kv, int page_shift) { return (key < kv ? key : kv - 1) >> page_shift; }

// Keys that some row at places p_lo .. p_hi sees: those up to p_hi that lie past
// `from` or are among the first `sinks`.
struct KeyRange {
  int from, to, sinks;
};
OCQ_HD KeyRange key_range(int p_lo, int p_hi, int window, int sinks) {
  return KeyRange{window > 0 && p_lo >= window ? p_lo - window : -1, p_hi, sinks};
}
// A row is read if its page is there and some row sees it; else it is taken as
// zeros: what lies in rows that no token sees (past the context, behind a
// window) never reaches a sum.
OCQ_HD bool page_there(int id, int num_pages) { return id >= 0 && id < num_pages; }
OCQ_HD bool key_in(int key, const KeyRange& k) { return key <= k.to && (key > k.from || key < k.sinks); }

// Offset of a key's row in the pool, without the head's part.  The entry
// points hold page strides below 2^32 and a page's rows within 2^31.
OCQ_HD uint64_t row_offset(int key, int id, int page_shift, uint32_t page, uint32_t token) {
  return (uint64_t)(uint32_t)id * page + (uint32_t)(key & ((1 << page_shift) - 1)) * token;
}

// Pieces.  Where every request's rows fit one row tile, the key tiles of each
// (request, kv head) are cut into pieces of about `per` tiles and each piece is
// one workgroup's work: as many pieces as the GPU holds workgroups at once,
// whatever the contexts' lengths, which only the device knows.
// Pieces of a request with T tiles (inv = 1 / per, rounded: any error moves
// only the number), and the tiles of piece i of c.
OCQ_HD int piece_count(int T, float inv) {
  const float x = (float)T * inv;
  int c = (int)x;
  c += (float)c < x;
  return T <= 0 ? 0 : c < 1 ? 1 : c > T ? T : c;
}
OCQ_HD int piece_begin(int T, int i, int c) { return (int)((int64_t)T * i / c); }
// Tiles per piece that are enough for `slots` pieces of `segments` segments
// with `total` tiles in all: sum of ceil(T / per) <= total / per + segments.
OCQ_HD int piece_bound(int total, int segments, int slots) { return total / (slots - segments) + 1; }

}  // namespace ocq
