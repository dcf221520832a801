// Attention of each request's new tokens over its paged cache.
//
// A row is one (token, query head); the rows of one request and kv head share
// its keys, so they are tiled together: row = token * group + head in group.
// Key j of the request is visible to the token at place p iff j <= p, j <
// kv_len and (no window, or j > p - window, or j < sinks).  With s_j = scale
// q.k_j the output is sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), in one pass
// over the keys with a running maximum m.
//
// Matrix form, for a tile of MT rows (MFMA 16x16x32 or 32x32x16, fp32 sums):
//   S^T = K Q^T    a lane holds row r = lane % MT and, of each key tile, keys
//                  8 (i / 4) + 4 (lane / MT) + i % 4;
//   O^T += V^T P^T the same registers, rounded to bf16, are already the
//                  second operand: only the order in which a step's keys are
//                  summed is fixed by the layout, and V is read in that order.
// Row statistics and the output's rescaling stay within a lane.  K and V come
// by direct-to-LDS loads into a ring of NST stages (16-byte chunks of a row
// xor-swizzled by the row, so that both the row reads of K and the transposing
// reads of V spread over the banks); V^T fragments come from LDS through the
// transposing reads.  E4M3 codes are converted exactly to bf16; the scale of a
// key multiplies its score, the scale of a value its probability.
//
// The maximum moves only when a score exceeds it by 2^8 (in the exponent of
// 2): probabilities up to 256 are as exact in bf16 and fp32 as those up to 1,
// and most tiles then need neither a cross-lane maximum nor a rescaling.
#include "gemm_core.h"
#include "layer_dev.h"
#include "layer_index.h"

#include <type_traits>

namespace ocq {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v2i lds_v2i;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLow = -3.4028234663852886e38f;   // below every score that is visible
constexpr float kSlack = 8.0f;                    // see above

constexpr int kTargetGroups = 512, kMinTiles = 4, kMaxSplits = 256;   // see plan_of
constexpr int kEvenRequests = 256;                // requests of a batch shared out evenly

// what a table entry outside the pool reads as
__device__ const v4i g_zero[1] = {};

// eight E4M3 codes -> bf16, exact (unit scale)
__device__ __forceinline__ v8bf e4m3x8_to_bf16(uint32_t lo, uint32_t hi) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int MT> struct Acc;
template <> struct Acc<16> { typedef v4f T; };
template <> struct Acc<32> { typedef v16f T; };

__device__ __forceinline__ v4f mfma(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v16f mfma(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// D: head size; KV8: E4M3 cache; MT x RT: rows of a wave, RT tiles of MT; WR x
// WK waves: over the rows and over the keys; TK: keys of a wave's stage; NST:
// stages; MINW: waves per SIMD that the registers leave room for.
template <int D_, bool KV8_, int MT_, int RT_, int WR_, int WK_, int TK_, int NST_, int MINW_>
struct Geo {
  static constexpr int RT = RT_, MINW = MINW_;
  static constexpr int D = D_, MT = MT_, WR = WR_, WK = WK_, TK = TK_, NST = NST_;
  static constexpr bool KV8 = KV8_;
  static constexpr int NW = WR * WK, THREADS = 64 * NW, ROWS = MT * RT * WR;
  static constexpr int ESZ = KV8 ? 1 : 2, RB = D * ESZ, CH = RB / 16;   // bytes and chunks of a row
  static constexpr int PART = TK * RB;                                  // K (or V) bytes of a key group's stage
  static constexpr int SCB = KV8 ? 2 * TK * 4 : 0;                      // its scales, K's then V's
  static constexpr int IDO = 2 * PART + SCB, STG = IDO + 256, RING = WK * NST * STG;   // 64 page ids at IDO
  static constexpr int QI = PART / 1024 / WR;                           // K (or V) loads per wave and stage
  static constexpr int SI = KV8 ? (2 * TK / 64 + WR - 1) / WR : 0;      // scale loads per wave and stage
  static constexpr int PW = 2 * QI + SI + 1;
  static constexpr int TT = TK * WK;                                    // keys of a tile, all key groups
  static constexpr int NKT = TK / MT;                                   // key tiles of a stage
  static constexpr int KS = 512 / MT;                                   // inputs of one MFMA (32 or 16)
  static constexpr int QS = D / KS, DT = D / MT, LG = 64 / MT;          // steps of S, tiles of O, lane groups
  static constexpr int PS = TK / KS;                                    // steps of O
  static constexpr int JOIN = WK > 1 ? WK * ROWS * (D * 4 + 8) : 0;
  static constexpr int LDS = RING > JOIN ? RING : JOIN;
  static constexpr bool EVEN = ROWS <= 64;                              // see layer_index.h, pieces
  static constexpr int RESIDENT = 256 * (MINW > 1 && LDS <= 78 * 1024 ? 2 : 1);   // workgroups at once, 256 CUs
  static_assert(PART % (1024 * WR) == 0 && TK % 32 == 0 && LDS <= 160 * 1024 && PW * (WR > 1 ? NST - 2 : NST - 1) < 64, "");
  static_assert(!KV8 || 2 * TK >= 64, "whole scale loads");
};

// Chunk swizzle: chunk c of row `row` lies at chunk c ^ swz(row).  What one
// pass of the banks (256 bytes) takes has to lie in different banks:
//   K   16 rows (16-byte reads), one chunk of each: swz takes 16 values over
//       16 rows, or 16 RB / 256 where a pass holds several rows;
//   V   half a wave's transposing reads: for bf16 4 rows x 4 chunks (MT 32) or
//       8 rows x 2 chunks (MT 16) from row 0 or 4 g, for codes 4 + 4 rows KB
//       apart x 2 chunks, or 8 + 8 rows x 1 chunk.
// So the row bits of V's pass go to the chunk bits above those it reads
// together.  Linear in the bits (swz(a + b) = swz(a) ^ swz(b) without carries).
template <class G>
__device__ __forceinline__ constexpr int swz(int row) {
  const int b0 = row & 1, b1 = row >> 1 & 1, b2 = row >> 2 & 1, b3 = row >> 3 & 1, b4 = row >> 4 & 1;
  if constexpr (!G::KV8) {
    if constexpr (G::MT == 32)
      return G::CH >= 16 ? b0 << 2 | b1 << 3 | b2 | b3 << 1 : b1 << 2 | b2 | b3 << 1;
    else
      return G::CH >= 16 ? b0 << 1 | b1 << 2 | b2 << 3 | b3 : b1 << 1 | b2 << 2 | b3;
  } else {
    if constexpr (G::MT == 32)
      return G::CH >= 16 ? b0 << 1 | b1 << 2 | b3 << 3 | b2 : G::CH == 8 ? b1 << 1 | b3 << 2 | b2 : b3 << 1 | b2;
    else
      return G::CH >= 16 ? b0 | b1 << 1 | b2 << 2 | (b3 ^ b4) << 3
             : G::CH == 8 ? b1 | b2 << 1 | (b3 ^ b4) << 2 : b2 | (b3 ^ b4) << 1;
  }
}

// p, or sixteen zero bytes; chosen by selects (a branch around each load would
// cost more than the load)
__device__ __forceinline__ const void* ok_or_zero(bool ok, const void* p) {
  uint64_t u = ok ? (uint64_t)p : (uint64_t)g_zero;
  asm("" : "+v"(u));
  return (const void*)u;
}

// Four V^T fragments (eight keys of one d per lane each) through the
// transposing LDS reads, at byte offset OFF from each address, in one block
// with its wait: the compiler would hold a builtin read back until every
// direct-to-LDS load of the wave has landed, the next stages' too.  The MFMAs
// of the block before run meanwhile.
template <int O0, int O1, int O2, int O3>
__device__ __forceinline__ void read_tr16(v2i (&x)[8], const uint32_t (&ad)[8]) {
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8 offset:%16\n\tds_read_b64_tr_b16 %1, %9 offset:%16\n\t"
      "ds_read_b64_tr_b16 %2, %10 offset:%17\n\tds_read_b64_tr_b16 %3, %11 offset:%17\n\t"
      "ds_read_b64_tr_b16 %4, %12 offset:%18\n\tds_read_b64_tr_b16 %5, %13 offset:%18\n\t"
      "ds_read_b64_tr_b16 %6, %14 offset:%19\n\tds_read_b64_tr_b16 %7, %15 offset:%19\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
      : "v"(ad[0]), "v"(ad[1]), "v"(ad[2]), "v"(ad[3]), "v"(ad[4]), "v"(ad[5]), "v"(ad[6]), "v"(ad[7]), "n"(O0),
        "n"(O1), "n"(O2), "n"(O3));
}
template <int O0, int O1, int O2, int O3>
__device__ __forceinline__ void read_tr8(v2i (&x)[4], const uint32_t (&ad)[4]) {
  asm volatile(
      "ds_read_b64_tr_b8 %0, %4 offset:%8\n\tds_read_b64_tr_b8 %1, %5 offset:%9\n\t"
      "ds_read_b64_tr_b8 %2, %6 offset:%10\n\tds_read_b64_tr_b8 %3, %7 offset:%11\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
      : "v"(ad[0]), "v"(ad[1]), "v"(ad[2]), "v"(ad[3]), "n"(O0), "n"(O1), "n"(O2), "n"(O3));
}

template <int N, class F>
__device__ __forceinline__ void unrolled(F f) {   // f(0) .. f(N - 1) with compile-time arguments
  if constexpr (N > 0) {
    unrolled<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// d of element j = 0 of a lane's operand in step s of S
template <class G>
__device__ __forceinline__ int q_dim(int s, int g) {
  if constexpr (G::KV8) return 2 * G::KS * (s >> 1) + 16 * g + 8 * (s & 1);   // one 16-byte read serves two steps
  else return G::KS * s + 8 * g;
}

// Inclusive sums over the lanes: within rows of 16 (DPP row_shr 1, 2, 4, 8),
// then each row's last into the next rows (row_bcast 15 and 31).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// The request that a workgroup (or a segment of the join) belongs to.
struct Found {
  int req, t0, n, kv;   // request (-1: none), its first new token, their number, its cached tokens
  int tiles, pieces;    // of each of its segments
  int first;            // its first piece (kv head 0)
};

// Every wave cuts the batch into pieces by itself, in registers: lane l holds
// request base + l.  of_piece >= 0: the request of that piece; else: request
// of_request.
__device__ __forceinline__ Found find_piece(const AttnArgs& a, int TT, int of_piece, int of_request) {
  const int lane = threadIdx.x & 63, kvh = a.c.kv_heads;
  auto load = [&](int base, int& t0, int& n, int& kv) {
    const int r = base + lane;
    t0 = n = kv = 0;
    if (r >= a.b.requests) return 0;
    const Span s = token_span(a.b.q_start, r, a.b.tokens);
    t0 = s.t0;
    n = s.n;
    kv = kv_bound(a.b.kv_lens[r], a.b.max_pages, a.c.page_shift);
    if (n <= 0) return 0;
    const int T = key_tiles(kv - n, kv - 1, a.window, a.sinks, TT).total;
    return T > 1 ? T : 1;   // a request without keys has its zeros to write
  };
  int t0, n, kv, T = load(0, t0, n, kv), total = T;
  for (int base = 64; base < a.b.requests; base += 64) {
    int x, y, z;
    total += load(base, x, y, z);
  }
  total = __builtin_amdgcn_readlane(wave_scan(total), 63) * kvh;
  const int segments = a.b.requests * kvh;
  float per;
  if (2 * segments > a.slots) {
    // about as many segments as slots: pieces of half a slot's share, so that
    // the last ones to run are short
    per = (float)(total / (2 * a.slots) + 1);
  } else {
    // the smallest pieces that fit the slots: eight candidates from the mean to
    // the bound, each summed by eight lanes
    const int lo = total / a.slots + 1, hi = piece_bound(total, segments, a.slots);
    per = (float)hi;
    if (a.b.requests <= 64) {
      const float mine = (float)lo + (float)(hi - lo) * (float)(lane >> 3) * 0.125f;
      const float inv = 1.0f / mine;
      int sum = 0;
      for (int r = lane & 7; r - (lane & 7) < a.b.requests; r += 8) sum += piece_count(__shfl(T, r), inv);
      sum += __builtin_amdgcn_update_dpp(0, sum, 0xB1, 0xF, 0xF, false);    // lane ^ 1
      sum += __builtin_amdgcn_update_dpp(0, sum, 0x4E, 0xF, 0xF, false);    // lane ^ 2
      sum += __builtin_amdgcn_update_dpp(0, sum, 0x141, 0xF, 0xF, false);   // 7 - lane of each eight
      const uint64_t fits = __ballot(sum * kvh <= a.slots);
      if (fits) per = __shfl(mine, __builtin_ctzll(fits));
    }
  }
  per = fmaxf(per, (float)kMinTiles);
  const float inv = 1.0f / per;
  Found f{-1, 0, 0, 0, 0, 0, 0};
  int carry = 0;
  for (int base = 0; base < a.b.requests; base += 64) {
    if (base > 0) T = load(base, t0, n, kv);
    const int c = piece_count(T, inv), end = wave_scan(c * kvh) + carry;
    // the lane whose request it is
    const bool mine = of_piece >= 0 ? of_piece < end && of_piece >= end - c * kvh : base + lane == of_request;
    const uint64_t who = __ballot(mine);
    if (who) {
      const int l = __builtin_ctzll(who);
      f.req = base + l;
      f.t0 = __builtin_amdgcn_readlane(t0, l);
      f.n = __builtin_amdgcn_readlane(n, l);
      f.kv = __builtin_amdgcn_readlane(kv, l);
      f.tiles = __builtin_amdgcn_readlane(T, l);
      f.pieces = __builtin_amdgcn_readlane(c, l);
      f.first = __builtin_amdgcn_readlane(end, l) - f.pieces * kvh;
      break;
    }
    carry = __builtin_amdgcn_readlane(end, 63);
  }
  return f;
}

// What a workgroup does next: stages s0 .. s1 of the key tiles of one row tile
// of one request and kv head.
struct Piece {
  int req, kvh, row0;   // first row of the tile
  int t0, n, kv, base;  // first new token, their number, cached tokens, place of the first new token
  int p_lo, p_hi;       // places of the tile's first and last rows
  KeyTiles tiles;
  int s0, s1;
  bool direct;          // the rows' whole result, or a part of it that goes to `part`
  size_t part;
};

template <class G>
__device__ __forceinline__ void attend(const AttnArgs& a, const Piece& pc, uint8_t* lds) {
  typedef typename Acc<G::MT>::T acc_t;
  constexpr int AN = G::MT == 16 ? 4 : 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave % G::WR, wk = wave / G::WR;
  const int r = lane % G::MT, g = lane / G::MT;
  const int n = pc.n, t0 = pc.t0, kv = pc.kv, base = pc.base, row0 = pc.row0, kvh = pc.kvh;
  const int p_lo = pc.p_lo, p_hi = pc.p_hi, ns = pc.s1 - pc.s0;

  // this lane's rows
  const int rl0 = wr * G::MT * G::RT + r;                    // in the tile; the next ones MT apart
  int place[G::RT];
  size_t at[G::RT];                                         // row of the output
  v8bf q[G::RT][G::QS];
#pragma unroll
  for (int t = 0; t < G::RT; ++t) {
    const int row = row0 + rl0 + t * G::MT;
    const bool live = row < n * a.group;
    const int tok = live ? row / a.group : 0, head = kvh * a.group + (live ? row % a.group : 0);
    place[t] = live ? base + tok : -1;
    at[t] = (size_t)(t0 + tok) * a.heads + head;
    const uint16_t* qp = a.q + (t0 + tok) * a.q_token + head * a.q_head;
#pragma unroll
    for (int s = 0; s < G::QS; ++s) {
      const v4i u = live ? *(const v4i*)(qp + q_dim<G>(s, g)) : v4i{0, 0, 0, 0};
      q[t][s] = __builtin_bit_cast(v8bf, u);
    }
  }
  const float c = a.scale * kLog2e;

  // ---- loads: rows of this wave's part of its key group's stage
  uint8_t* const ring = lds + wk * (G::NST * G::STG);
  const int32_t* const table = a.b.table + pc.req * a.b.table_stride;
  const uint8_t* const k_head = a.c.k + kvh * a.c.head;
  const uint8_t* const v_head = a.c.v + kvh * a.c.head;
  const float* const ks_head = a.c.k_scale + (G::KV8 ? kvh * a.c.s_head : 0);
  const float* const vs_head = a.c.v_scale + (G::KV8 ? kvh * a.c.s_head : 0);
  // first key of the wave's key group in stage st
  auto tile_key = [&](int st) { return tile_of(pc.tiles, pc.s0 + st) * G::TT + wk * G::TK; };
  constexpr int AHEAD = G::WR > 1 ? G::NST - 1 : G::NST;   // stages on their way, see the ring below
  auto q_row = [&](int i) { return ((i * G::WR + wr) * 64 + lane) / G::CH; };          // row of load i
  auto sc_key = [&](int i) { return (((i * G::WR + wr) * 64 + lane) % (2 * G::TK)) % G::TK; };   // key of scale load i
  // Page ids come with the stage AHEAD before the one that they are for: a
  // load into registers would have to be waited for together with every
  // earlier load of the wave.
  auto entry = [&](int st, int row) { return table + table_entry(tile_key(st) + row, kv, a.c.page_shift); };
  auto issue = [&](int st, uint8_t* slot, auto id_of) {
    const int key0 = tile_key(st);
    int ids[G::QI + G::SI];
#pragma unroll
    for (int i = 0; i < G::QI + G::SI; ++i) ids[i] = id_of(i < G::QI ? q_row(i) : sc_key(i - G::QI));
    const int later = st + AHEAD < ns ? st + AHEAD : st;
    __builtin_amdgcn_global_load_lds((const void*)entry(later, lane % G::TK), (lds_void*)(slot + G::IDO), 4, 0, 0);
#pragma unroll
    for (int i = 0; i < G::QI; ++i) {
      const int rw = q_row(i), key = key0 + rw, lin = ((i * G::WR + wr) * 64 + lane) % G::CH;
      const bool ok = row_there(key, kv, ids[i], a.c.num_pages);
      const uint64_t off = row_offset(key, ids[i], a.c.page_shift, a.c.page, a.c.token) + ((lin ^ swz<G>(rw)) << 4);
      uint8_t* dst = slot + (i * G::WR + wr) * 1024;
      __builtin_amdgcn_global_load_lds(ok_or_zero(ok, k_head + off), (lds_void*)dst, 16, 0, 0);
      __builtin_amdgcn_global_load_lds(ok_or_zero(ok, v_head + off), (lds_void*)(dst + G::PART), 16, 0, 0);
    }
    if constexpr (G::KV8) {
#pragma unroll
      for (int i = 0; i < G::SI; ++i) {
        const int lin = ((i * G::WR + wr) * 64) % (2 * G::TK);   // where this load's 64 scales go
        const int key = key0 + sc_key(i);
        const bool ok = row_there(key, kv, ids[G::QI + i], a.c.num_pages);
        const uint64_t off = row_offset(key, ids[G::QI + i], a.c.page_shift, a.c.s_page, a.c.s_token);
        const float* src = (lin + lane >= G::TK ? vs_head : ks_head) + off;
        __builtin_amdgcn_global_load_lds(ok_or_zero(ok, src), (lds_void*)(slot + 2 * G::PART + lin * 4), 4, 0, 0);
      }
    }
  };

  acc_t o[G::RT][G::DT];
  float m[G::RT], l[G::RT];
#pragma unroll
  for (int t = 0; t < G::RT; ++t) {
    m[t] = kLow;
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < G::DT; ++d)
#pragma unroll
      for (int i = 0; i < AN; ++i) o[t][d][i] = 0.0f;
  }

  // where the lane's part of a V^T fragment lies in a stage: tile d of the
  // output, keys kb + 4 g + {0..3} (first half) and kb + KB + 4 g + {0..3}
  uint32_t v_off[G::DT][G::KV8 ? 1 : 2];
  {
    constexpr int KB = G::MT == 16 ? 16 : 8;
    const int i16 = lane & 15, dh = G::MT == 32 ? ((lane >> 4) & 1) * 16 : 0;
#pragma unroll
    for (int d = 0; d < G::DT; ++d)
#pragma unroll
      for (int h = 0; h < (G::KV8 ? 1 : 2); ++h) {
        const int key = G::KV8 ? (i16 >> 3) * KB + 4 * g + ((i16 >> 1) & 3) : h * KB + 4 * g + (i16 >> 2);
        const int ch = G::KV8 ? (d * G::MT + dh) / 16 : (d * G::MT + dh) / 8 + ((i16 >> 1) & 1);
        v_off[d][h] = key * G::RB + ((ch ^ swz<G>(key)) << 4) + 8 * (i16 & 1);
      }
  }

  // ---- one stage
  auto compute = [&](int st, const uint8_t* slot) {
    const int key0 = tile_key(st);
    acc_t s[G::RT][G::NKT];
#pragma unroll
    for (int kt = 0; kt < G::NKT; ++kt) {
#pragma unroll
      for (int t = 0; t < G::RT; ++t)
#pragma unroll
        for (int i = 0; i < AN; ++i) s[t][kt][i] = 0.0f;
      const uint8_t* kr = slot + (kt * G::MT + r) * G::RB;
      const int f = swz<G>(r) ^ swz<G>(kt * G::MT);
      if constexpr (!G::KV8) {
        v8bf ka[G::QS];
#pragma unroll
        for (int x = 0; x < G::QS; ++x) ka[x] = *(const v8bf*)(kr + (((x * G::LG + g) ^ f) << 4));
        __builtin_amdgcn_sched_barrier(0);   // every read on its way before the first product waits
#pragma unroll
        for (int x = 0; x < G::QS; ++x)
#pragma unroll
          for (int t = 0; t < G::RT; ++t) s[t][kt] = mfma(ka[x], q[t][x], s[t][kt]);
      } else {
        v4i ku[G::QS / 2];
#pragma unroll
        for (int x = 0; x < G::QS; x += 2) ku[x / 2] = *(const v4i*)(kr + (((x / 2 * G::LG + g) ^ f) << 4));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < G::QS; x += 2) {
          const v4i u = ku[x / 2];
          const v8bf k0 = e4m3x8_to_bf16(u[0], u[1]), k1 = e4m3x8_to_bf16(u[2], u[3]);
#pragma unroll
          for (int t = 0; t < G::RT; ++t) {
            s[t][kt] = mfma(k0, q[t][x], s[t][kt]);
            s[t][kt] = mfma(k1, q[t][x + 1], s[t][kt]);
          }
        }
      }
    }
    const float* sc = (const float*)(slot + 2 * G::PART);
    const bool whole = key0 + G::TK - 1 <= p_lo && (a.window <= 0 || key0 > p_hi - a.window);
    uint32_t p[G::RT][G::NKT * AN / 2];
#pragma unroll
    for (int t = 0; t < G::RT; ++t) {
#pragma unroll
      for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
        for (int i4 = 0; i4 < AN / 4; ++i4) {
          const int kk = kt * G::MT + 8 * i4 + 4 * g;   // first of four keys
          v4f ks = {1.0f, 1.0f, 1.0f, 1.0f};
          if constexpr (G::KV8) ks = *(const v4f*)(sc + kk);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = s[t][kt][4 * i4 + i];
            if constexpr (G::KV8) x *= ks[i];
            s[t][kt][4 * i4 + i] = x;
          }
        }
      if (!whole) {
#pragma unroll
        for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
          for (int i = 0; i < AN; ++i) {
            const int j = key0 + kt * G::MT + 8 * (i >> 2) + 4 * g + (i & 3);
            s[t][kt][i] = key_seen(j, place[t], a.window, a.sinks) ? s[t][kt][i] : -__builtin_inff();
          }
      }
      float top = -__builtin_inff();
#pragma unroll
      for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
        for (int i = 0; i < AN; ++i) top = fmaxf(top, s[t][kt][i]);
      // scores in the exponent of 2 from here on: c s - m
      if (__any(top * c > m[t] + kSlack)) {
        float nm = top * c;
#pragma unroll
        for (int x = G::MT; x < 64; x <<= 1) nm = fmaxf(nm, __shfl_xor(nm, x));
        nm = fmaxf(nm, m[t]);
        const float f = __builtin_amdgcn_exp2f(m[t] - nm);
        m[t] = nm;
        l[t] *= f;
#pragma unroll
        for (int d = 0; d < G::DT; ++d)
#pragma unroll
          for (int i = 0; i < AN; ++i) o[t][d][i] *= f;
      }
#pragma unroll
      for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
        for (int i4 = 0; i4 < AN / 4; ++i4) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][kt][4 * i4 + i], c, -m[t]));
            l[t] += e[i];
          }
          if constexpr (G::KV8) {
            const v4f vs = *(const v4f*)(sc + G::TK + kt * G::MT + 8 * i4 + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] *= vs[i];
          }
          p[t][(kt * AN + 4 * i4) / 2] = pack_bf16(e[0], e[1]);
          p[t][(kt * AN + 4 * i4) / 2 + 1] = pack_bf16(e[2], e[3]);
        }
    }
    // O^T += V^T P^T, four fragments (step x of the keys, tile d of the output) at a time
    const uint32_t sb = (uint32_t)(uintptr_t)(lds_void*)slot;
    unrolled<G::PS * G::DT / 4>([&](auto blk) {
      constexpr int F0 = 4 * decltype(blk)::value;
      auto off = [](int f) constexpr { return G::PART + f / G::DT * G::KS * G::RB; };
      v8bf va[4];
      if constexpr (!G::KV8) {
        uint32_t ad[8];
        v2i x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) ad[j] = sb + v_off[(F0 + j / 2) % G::DT][j & 1];
        read_tr16<off(F0), off(F0 + 1), off(F0 + 2), off(F0 + 3)>(x, ad);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          va[j] = __builtin_bit_cast(v8bf, __builtin_shufflevector(x[2 * j], x[2 * j + 1], 0, 1, 2, 3));
      } else {
        uint32_t ad[4];
        v2i x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) ad[j] = sb + v_off[(F0 + j) % G::DT][0];
        read_tr8<off(F0), off(F0 + 1), off(F0 + 2), off(F0 + 3)>(x, ad);
#pragma unroll
        for (int j = 0; j < 4; ++j) va[j] = e4m3x8_to_bf16((uint32_t)x[j][0], (uint32_t)x[j][1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        constexpr int DT = G::DT;
        const int x = (F0 + j) / DT, d = (F0 + j) % DT;
#pragma unroll
        for (int t = 0; t < G::RT; ++t) {
          const v8bf pb = __builtin_bit_cast(
              v8bf, (v4i{(int)p[t][4 * x], (int)p[t][4 * x + 1], (int)p[t][4 * x + 2], (int)p[t][4 * x + 3]}));
          o[t][d] = mfma(va[j], pb, o[t][d]);
        }
      }
    });
  };

  // ---- the ring.  Waves that share a stage meet once for it: then its loads
  // have landed and stage st - 1 is done with, so stage st + NST - 1 goes where
  // that was.  A wave alone refills a slot as soon as it has read it, so that
  // NST stages are on their way while it waits.
  if (ns > 0) {
#pragma unroll
    for (int st = 0; st < AHEAD; ++st)
      if (st < ns) issue(st, ring + st * G::STG, [&](int row) { return *entry(st, row); });
    int slot = 0;
    for (int st = 0; st < ns; ++st) {
      uint8_t* const at_st = ring + slot * G::STG;
      // stage st has landed once at most the later ones' loads are outstanding
      if (st + AHEAD - 1 < ns) wait_vm<(AHEAD - 1) * G::PW>();
      else wait_vm<0>();
      auto next = [&](uint8_t* to) {
        issue(st + AHEAD, to, [&](int row) { return *(const int*)(at_st + G::IDO + 4 * row); });
      };
      if constexpr (G::WR > 1) {
        lds_barrier();
        if (st + AHEAD < ns) next(ring + (slot == 0 ? G::NST - 1 : slot - 1) * G::STG);
        compute(st, at_st);
      } else {
        asm volatile("" ::: "memory");
        compute(st, at_st);
        if (st + AHEAD < ns) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          next(at_st);
        }
      }
      slot = slot + 1 == G::NST ? 0 : slot + 1;
    }
  }

  // ---- join the lane groups' sums and the key groups' parts, and write
#pragma unroll
  for (int t = 0; t < G::RT; ++t)
#pragma unroll
    for (int x = G::MT; x < 64; x <<= 1) l[t] += __shfl_xor(l[t], x);
  // where row rl of the tile (row `at` of the output) goes if it is a part
  auto part_at = [&](int rl, size_t at) { return pc.part + (a.even ? (size_t)rl : at); };
  if constexpr (G::WK == 1) {
#pragma unroll
    for (int t = 0; t < G::RT; ++t) {
      if (row0 + rl0 + t * G::MT >= n * a.group) continue;
      const float inv = l[t] > 0.0f ? 1.0f / l[t] : l[t];   // l: 0, or NaN kept
      const float lse2 = l[t] == 0.0f ? -__builtin_inff() : m[t] + __builtin_amdgcn_logf(l[t]);
      const size_t ps = part_at(rl0 + t * G::MT, at[t]);
#pragma unroll
      for (int d = 0; d < G::DT; ++d)
#pragma unroll
        for (int i4 = 0; i4 < AN / 4; ++i4) {
          const int d4 = d * G::MT + 8 * i4 + 4 * g;
          const v4f y = {o[t][d][4 * i4] * inv, o[t][d][4 * i4 + 1] * inv, o[t][d][4 * i4 + 2] * inv,
                         o[t][d][4 * i4 + 3] * inv};
          if (pc.direct)
            *(v2i*)(a.out + at[t] * G::D + d4) = v2i{(int)pack_bf16(y[0], y[1]), (int)pack_bf16(y[2], y[3])};
          else if (ns > 0)
            *(v4f*)(a.part_o + ps * G::D + d4) = y;
        }
      if (g == 0 && pc.direct && a.lse) a.lse[at[t]] = lse2 * kLn2;
      if (g == 0 && !pc.direct) a.part_lse[ps] = lse2;
    }
  } else {
    float* const so = (float*)lds;                          // [WK][ROWS][D]
    float* const sm = so + G::WK * G::ROWS * G::D;          // [2][WK][ROWS]: m, l
    __syncthreads();                                        // the ring is no longer read
#pragma unroll
    for (int t = 0; t < G::RT; ++t) {
      const int rl = rl0 + t * G::MT;
      if (g == 0) {
        sm[wk * G::ROWS + rl] = m[t];
        sm[(G::WK + wk) * G::ROWS + rl] = l[t];
      }
#pragma unroll
      for (int d = 0; d < G::DT; ++d)
#pragma unroll
        for (int i4 = 0; i4 < AN / 4; ++i4)
          *(v4f*)(so + (wk * G::ROWS + rl) * G::D + d * G::MT + 8 * i4 + 4 * g) =
              v4f{o[t][d][4 * i4], o[t][d][4 * i4 + 1], o[t][d][4 * i4 + 2], o[t][d][4 * i4 + 3]};
    }
    __syncthreads();
    constexpr int LPR = G::D / 4;                           // lanes per row, 4 values each
    for (int it = threadIdx.x; it < G::ROWS * LPR; it += G::THREADS) {
      const int rw = it / LPR, d = (it % LPR) * 4, rg = row0 + rw;
      if (rg >= n * a.group) break;
      float mm = kLow;
#pragma unroll
      for (int x = 0; x < G::WK; ++x) mm = fmaxf(mm, sm[x * G::ROWS + rw]);
      float ll = 0.0f;
      v4f ov = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < G::WK; ++x) {
        const float f = __builtin_amdgcn_exp2f(sm[x * G::ROWS + rw] - mm);
        ll += sm[(G::WK + x) * G::ROWS + rw] * f;
        const v4f y = *(const v4f*)(so + (x * G::ROWS + rw) * G::D + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) ov[i] += y[i] * f;
      }
      const float inv = ll > 0.0f ? 1.0f / ll : ll;
      const float lse2 = ll == 0.0f ? -__builtin_inff() : mm + __builtin_amdgcn_logf(ll);
      const size_t ar = a.even && !pc.direct ? 0 : (size_t)(t0 + rg / a.group) * a.heads + kvh * a.group + rg % a.group;
      if (pc.direct) {
        *(v2i*)(a.out + ar * G::D + d) = v2i{(int)pack_bf16(ov[0] * inv, ov[1] * inv),
                                             (int)pack_bf16(ov[2] * inv, ov[3] * inv)};
        if (d == 0 && a.lse) a.lse[ar] = lse2 * kLn2;
      } else {
        const size_t ps = part_at(rw, ar);
        if (ns > 0) *(v4f*)(a.part_o + ps * G::D + d) = v4f{ov[0] * inv, ov[1] * inv, ov[2] * inv, ov[3] * inv};
        if (d == 0) a.part_lse[ps] = lse2;
      }
    }
  }
}

template <class G>
__global__ __launch_bounds__(G::THREADS, G::MINW) void k_attn(AttnArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  Piece pc;
  if constexpr (G::EVEN) {
    if (a.even) {
      const Found f = find_piece(a, G::TT, blockIdx.x, 0);
      if (f.req < 0) return;
      const int in = blockIdx.x - f.first, i = in % f.pieces;
      pc.req = f.req;
      pc.kvh = in / f.pieces;
      pc.row0 = 0;
      pc.t0 = f.t0;
      pc.n = f.n;
      pc.kv = f.kv;
      pc.base = pc.p_lo = f.kv - f.n;
      pc.p_hi = f.kv - 1;
      pc.tiles = key_tiles(pc.p_lo, pc.p_hi, a.window, a.sinks, G::TT);
      pc.s0 = pc.tiles.total ? piece_begin(f.tiles, i, f.pieces) : 0;
      pc.s1 = pc.tiles.total ? piece_begin(f.tiles, i + 1, f.pieces) : 0;
      pc.direct = f.pieces == 1;
      pc.part = (size_t)blockIdx.x * G::ROWS;
      attend<G>(a, pc, lds);
      return;
    }
  }
  // One row tile: pair (request, kv head) fastest, so that workgroups that
  // share keys are 8 apart where the pairs are a multiple of 8 and meet in one
  // XCD's L2; row tiles from the last (most keys) to the first.
  const int pairs = a.b.requests * a.c.kv_heads, pair = blockIdx.x % pairs;
  const int rest = blockIdx.x / pairs, split = rest % a.splits;
  const int tile = (int)(gridDim.x / pairs / a.splits) - 1 - rest / a.splits;
  pc.req = pair / a.c.kv_heads;
  pc.kvh = pair % a.c.kv_heads;
  const Span span = token_span(a.b.q_start, pc.req, a.b.tokens);
  pc.t0 = span.t0;
  pc.n = span.n;
  pc.row0 = tile * G::ROWS;
  if (span.n <= 0 || pc.row0 >= span.n * a.group) return;
  pc.kv = kv_bound(a.b.kv_lens[pc.req], a.b.max_pages, a.c.page_shift);
  pc.base = pc.kv - pc.n;
  const int last_row = (pc.row0 + G::ROWS < pc.n * a.group ? pc.row0 + G::ROWS : pc.n * a.group) - 1;
  pc.p_lo = pc.base + pc.row0 / a.group;
  pc.p_hi = pc.base + last_row / a.group;
  pc.tiles = key_tiles(pc.p_lo, pc.p_hi, a.window, a.sinks, G::TT);
  const int per = (pc.tiles.total + a.splits - 1) / a.splits;
  pc.s0 = split * per < pc.tiles.total ? split * per : pc.tiles.total;
  pc.s1 = pc.s0 + per < pc.tiles.total ? pc.s0 + per : pc.tiles.total;
  pc.direct = a.splits == 1;
  pc.part = (size_t)split * a.b.tokens * a.heads;
  attend<G>(a, pc, lds);
}

// sum_i 2^(lse_i - mm) out_i and ll = sum_i 2^(lse_i - mm) over the n parts of a
// row (part i at row_of(i)), mm the largest lse; a part without keys (lse
// -inf) has no output.  Eight parts are read at a time.
template <class F>
__device__ __forceinline__ v4f join_parts(const AttnArgs& a, int n, int d, int D, F row_of, float& mm, float& ll) {
  constexpr int B = 8;
  mm = -__builtin_inff();
  ll = 0.0f;
  v4f ov = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i0 = 0; i0 < n; i0 += B) {
    float x[B];
    v4f y[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const size_t r = row_of(i0 + j < n ? i0 + j : n - 1);
      x[j] = a.part_lse[r];
      y[j] = *(const v4f*)(a.part_o + r * D + d);
    }
    float nm = mm;
#pragma unroll
    for (int j = 0; j < B; ++j) {
      if (i0 + j >= n) x[j] = -__builtin_inff();
      nm = fmaxf(nm, x[j]);
    }
    if (nm == -__builtin_inff()) continue;   // nothing yet (NaN goes on)
    const float f = __builtin_amdgcn_exp2f(mm - nm);
    ll *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i) ov[i] *= f;
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const float e = __builtin_amdgcn_exp2f(x[j] - nm);
      ll += e;
#pragma unroll
      for (int i = 0; i < 4; ++i) ov[i] += x[j] == -__builtin_inff() ? 0.0f : y[j][i] * e;
    }
    mm = nm;
  }
  return ov;
}

// Joins the splits: out = sum_s 2^(lse_s - lse) out_s.  D / 4 lanes per row;
// a split without keys (lse -inf) has no output and is skipped.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int LPR = D / 4, RPB = 256 / LPR;
  const size_t rows = (size_t)a.b.tokens * a.heads;
  const size_t at = (size_t)blockIdx.x * RPB + threadIdx.x / LPR;
  const int d = (threadIdx.x % LPR) * 4;
  if (at >= rows) return;
  float ll, mm;
  const v4f ov = join_parts(a, a.splits, d, D, [&](int s) { return s * rows + at; }, mm, ll);
  const float inv = ll > 0.0f ? 1.0f / ll : ll;
  *(v2i*)(a.out + at * D + d) = v2i{(int)pack_bf16(ov[0] * inv, ov[1] * inv), (int)pack_bf16(ov[2] * inv, ov[3] * inv)};
  if (d == 0 && a.lse) a.lse[at] = ll == 0.0f ? -__builtin_inff() : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
}

// Joins the pieces of the segments that were cut.
template <class G>
__global__ __launch_bounds__(256) void k_attn_join_pieces(AttnArgs a) {
  constexpr int LPR = G::D / 4, RPB = 256 / LPR, BPS = G::ROWS / RPB;   // rows a block, blocks a segment
  const int pair = blockIdx.x / BPS, kvh = pair % a.c.kv_heads;
  const int rw = blockIdx.x % BPS * RPB + threadIdx.x / LPR, d = (threadIdx.x % LPR) * 4;
  const Found f = find_piece(a, G::TT, -1, pair / a.c.kv_heads);
  if (f.req < 0 || f.pieces <= 1 || rw >= f.n * a.group) return;
  auto slot = [&](int i) { return (size_t)(f.first + kvh * f.pieces + i) * G::ROWS + rw; };
  float ll, mm;
  const v4f ov = join_parts(a, f.pieces, d, G::D, slot, mm, ll);
  const float inv = ll > 0.0f ? 1.0f / ll : ll;
  const size_t at = (size_t)(f.t0 + rw / a.group) * a.heads + kvh * a.group + rw % a.group;
  *(v2i*)(a.out + at * G::D + d) =
      v2i{(int)pack_bf16(ov[0] * inv, ov[1] * inv), (int)pack_bf16(ov[2] * inv, ov[3] * inv)};
  if (d == 0 && a.lse) a.lse[at] = ll == 0.0f ? -__builtin_inff() : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
}

template <class G>
hipError_t run(const AttnArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const hipError_t e = allow_lds((const void*)k_attn<G>, G::LDS, allowed);
  if (e != hipSuccess) return e;
  const int pairs = a.b.requests * a.c.kv_heads;
  if (a.even) {
    hipLaunchKernelGGL((k_attn<G>), dim3(a.groups), dim3(G::THREADS), G::LDS, st, a);
    if constexpr (G::EVEN)
      hipLaunchKernelGGL((k_attn_join_pieces<G>), dim3(pairs * (G::ROWS * G::D / 1024)), dim3(256), 0, st, a);
    return hipGetLastError();
  }
  const int tiles = (int)(((int64_t)a.max_new * a.group + G::ROWS - 1) / G::ROWS);
  hipLaunchKernelGGL((k_attn<G>), dim3((unsigned)((int64_t)pairs * a.splits * tiles)), dim3(G::THREADS), G::LDS, st, a);
  if (a.splits > 1) {
    const size_t rows = (size_t)a.b.tokens * a.heads, rpb = 1024 / G::D;
    hipLaunchKernelGGL((k_attn_join<G::D>), dim3((unsigned)((rows + rpb - 1) / rpb)), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

// The kernel for a call whose largest request has `rows` rows per kv head.
// Up to 16 and 32 rows each wave takes all of them and a part of the keys,
// without barriers; up to 64, two waves share the keys of two; beyond, four
// waves of 32 rows share every key tile.  Key groups and stages fill the LDS.
template <int D, bool KV8, class F>
auto visit_rows(int64_t rows, F f) {
  if (rows <= 16) return f(Geo<D, KV8, 16, 1, 1, D == 256 && !KV8 ? 2 : 4, 32, 2, D == 256 ? 1 : 2>{});
  if constexpr (D < 256)
    if (rows <= 32) return f(Geo<D, KV8, 32, 1, 1, 4, 32, 2, 2>{});
  if (rows <= 64) return f(Geo<D, KV8, 32, 1, 2, 2, 32, 2, D == 256 ? 1 : 2>{});
  return f(Geo<D, KV8, 32, 1, 4, 1, D == 256 ? 32 : 64, 2, D == 256 ? 1 : 2>{});
}
template <class F>
auto visit(int dim, bool e4m3, int64_t rows, F f) {
  if (dim == 64) return e4m3 ? visit_rows<64, true>(rows, f) : visit_rows<64, false>(rows, f);
  if (dim == 128) return e4m3 ? visit_rows<128, true>(rows, f) : visit_rows<128, false>(rows, f);
  return e4m3 ? visit_rows<256, true>(rows, f) : visit_rows<256, false>(rows, f);
}

}  // namespace

// How a call is laid out.
//  * All rows of a request in one tile and more keys than one piece: pieces,
//    for two workgroups' worth of LDS (or one) on every CU.
//  * Several row tiles per request but few in all: each tile's keys in equal
//    splits, none below four key tiles of the longest request.
//  * Else one workgroup per row tile, all its keys: enough of them to fill the
//    GPU by themselves, or too few keys to be worth a second launch.
AttnPlan attn_plan(int tokens, int requests, int max_new, int max_kv, int heads, int kv_heads, int dim, int e4m3,
                   int window, int sinks, int64_t cap) {
  const int64_t rows = (int64_t)max_new * (heads / kv_heads);
  int64_t keys = max_kv;
  if (window > 0 && (int64_t)window + sinks + max_new < keys) keys = (int64_t)window + sinks + max_new;
  return visit(dim, e4m3 != 0, rows, [&](auto geo) {
    typedef decltype(geo) G;
    AttnPlan p{0, 1, 0, 0, 0};
    const int64_t pairs = (int64_t)requests * kv_heads, tiles = (rows + G::ROWS - 1) / G::ROWS;
    const int64_t key_tiles = (keys + G::TT - 1) / G::TT;
    if (key_tiles <= kMinTiles) return p;
    if (G::EVEN && requests <= kEvenRequests && pairs < 4 * G::RESIDENT && pairs * (cap / G::TT + 1) < (1 << 30)) {
      p.even = 1;
      p.slots = G::RESIDENT;
      p.groups = (int)(2 * pairs > p.slots ? 2 * p.slots + pairs : p.slots);   // no fewer than there can be pieces
      p.part_rows = (size_t)p.groups * G::ROWS;
      return p;
    }
    const int64_t groups = pairs * tiles, want = (kTargetGroups + groups - 1) / groups, most = key_tiles / kMinTiles;
    const int64_t s = want < most ? want : most;
    p.splits = (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
    p.part_rows = p.splits > 1 ? (size_t)p.splits * tokens * heads : 0;
    return p;
  });
}

int launch_attn(const AttnArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  return (int)visit(a.dim, a.e4m3 != 0, (int64_t)a.max_new * a.group,
                    [&](auto geo) { return run<decltype(geo)>(a, st); });
}

}  // namespace ocq
