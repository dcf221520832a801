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

constexpr int kTargetGroups = 512, kMinTiles = 4, kMaxSplits = 256;   // see attn_splits

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

// D: head size; KV8: E4M3 cache; MT: rows of a wave's tile; WR x WK waves:
// over the rows and over the keys; TK: keys of a wave's stage; NST: stages.
template <int D_, bool KV8_, int MT_, int WR_, int WK_, int TK_, int NST_>
struct Geo {
  static constexpr int D = D_, MT = MT_, WR = WR_, WK = WK_, TK = TK_, NST = NST_;
  static constexpr bool KV8 = KV8_;
  static constexpr int NW = WR * WK, THREADS = 64 * NW, ROWS = MT * WR;
  static constexpr int ESZ = KV8 ? 1 : 2, RB = D * ESZ, CH = RB / 16;   // bytes and chunks of a row
  static constexpr int PART = TK * RB;                                  // K (or V) bytes of a key group's stage
  static constexpr int SCB = KV8 ? 2 * TK * 4 : 0;                      // its scales, K's then V's
  static constexpr int STG = 2 * PART + SCB, RING = WK * NST * STG;
  static constexpr int QI = PART / 1024 / WR;                           // K (or V) loads per wave and stage
  static constexpr int SI = KV8 ? (2 * TK / 64 + WR - 1) / WR : 0;      // scale loads per wave and stage
  static constexpr int PW = 2 * QI + SI;
  static constexpr int TT = TK * WK;                                    // keys of a tile, all key groups
  static constexpr int NKT = TK / MT;                                   // key tiles of a stage
  static constexpr int KS = 512 / MT;                                   // inputs of one MFMA (32 or 16)
  static constexpr int QS = D / KS, DT = D / MT, LG = 64 / MT;          // steps of S, tiles of O, lane groups
  static constexpr int PS = TK / KS;                                    // steps of O
  static constexpr int MINW = D == 256 && MT == 32 ? 1 : 2;             // waves per SIMD the registers leave room for
  static constexpr int JOIN = WK > 1 ? WK * ROWS * (D * 4 + 8) : 0;
  static constexpr int LDS = RING > JOIN ? RING : JOIN;
  static_assert(PART % (1024 * WR) == 0 && TK % 32 == 0 && LDS <= 160 * 1024 && PW * (NST - 1) < 64, "");
  static_assert(!KV8 || 2 * TK >= 64, "whole scale loads");
};

// Chunk swizzle of row `row`: 256 bytes of LDS hold 256 / RB rows.
template <class G>
__device__ __forceinline__ constexpr int swz(int row) {
  return G::CH >= 16 ? row & 15 : G::CH == 8 ? (row >> 1) & 7 : (row >> 2) & 3;
}

// d of element j = 0 of a lane's operand in step s of S
template <class G>
__device__ __forceinline__ int q_dim(int s, int g) {
  if constexpr (G::KV8) return 2 * G::KS * (s >> 1) + 16 * g + 8 * (s & 1);   // one 16-byte read serves two steps
  else return G::KS * s + 8 * g;
}

template <class G>
__global__ __launch_bounds__(G::THREADS, G::MINW) void k_attn(AttnArgs a) {
  typedef typename Acc<G::MT>::T acc_t;
  constexpr int AN = G::MT == 16 ? 4 : 16;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave % G::WR, wk = wave / G::WR;
  const int r = lane % G::MT, g = lane / G::MT;

  // pair (request, kv head) fastest: workgroups that share keys are 8 apart
  // where the pairs are a multiple of 8, so they meet in one XCD's L2.  Row
  // tiles from the last (most keys) to the first.
  const int pairs = a.b.requests * a.c.kv_heads;
  const int pair = blockIdx.x % pairs, rest = blockIdx.x / pairs;
  const int split = rest % a.splits;
  const int tile = (int)(gridDim.x / pairs / a.splits) - 1 - rest / a.splits;
  const int req = pair / a.c.kv_heads, kvh = pair % a.c.kv_heads;
  const Span span = token_span(a.b.q_start, req, a.b.tokens);
  const int t0 = span.t0, n = span.n;
  const int row0 = tile * G::ROWS;
  if (n <= 0 || row0 >= n * a.group) return;
  const int kv = kv_bound(a.b.kv_lens[req], a.b.max_pages, a.c.page_shift);
  const int base = kv - n;                                  // place of the first new token
  const int last_row = (row0 + G::ROWS < n * a.group ? row0 + G::ROWS : n * a.group) - 1;
  const int p_lo = base + row0 / a.group, p_hi = base + last_row / a.group;
  const KeyTiles tiles = key_tiles(p_lo, p_hi, a.window, a.sinks, G::TT);
  const int per = (tiles.total + a.splits - 1) / a.splits;
  const int s0 = split * per < tiles.total ? split * per : tiles.total;
  const int s1 = s0 + per < tiles.total ? s0 + per : tiles.total;
  const int ns = s1 - s0;

  // this lane's row
  const int row = row0 + wr * G::MT + r;
  const bool live = row < n * a.group;
  const int tok = live ? row / a.group : 0, head = kvh * a.group + (live ? row % a.group : 0);
  const int place = live ? base + tok : -1;

  v8bf q[G::QS];
  {
    const uint16_t* qp = a.q + (t0 + tok) * a.q_token + head * a.q_head;
#pragma unroll
    for (int s = 0; s < G::QS; ++s) {
      const v4i u = live ? *(const v4i*)(qp + q_dim<G>(s, g)) : v4i{0, 0, 0, 0};
      q[s] = __builtin_bit_cast(v8bf, u);
    }
  }
  const float c = a.scale * kLog2e;

  // ---- loads: rows of this wave's part of its key group's stage
  uint8_t* const ring = lds + wk * (G::NST * G::STG);
  const int32_t* const table = a.b.table + req * a.b.table_stride;
  const int64_t head_off = kvh * a.c.head;
  // first key of the wave's key group in stage st
  auto tile_key = [&](int st) { return tile_of(tiles, s0 + st) * G::TT + wk * G::TK; };
  constexpr int kIds = G::QI + G::SI;
  int ids[kIds];
  auto q_row = [&](int i) { return ((i * G::WR + wr) * 64 + lane) / G::CH; };          // row of load i
  auto sc_key = [&](int i) { return (((i * G::WR + wr) * 64 + lane) % (2 * G::TK)) % G::TK; };   // key of scale load i
  auto fetch_ids = [&](int st) {
    const int key0 = tile_key(st);
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      const int key = key0 + (i < G::QI ? q_row(i) : sc_key(i - G::QI));
      ids[i] = table[table_entry(key, kv, a.c.page_shift)];
    }
  };
  auto issue = [&](int st, uint8_t* slot) {
    const int key0 = tile_key(st);
#pragma unroll
    for (int i = 0; i < G::QI; ++i) {
      const int rw = q_row(i), key = key0 + rw, lin = ((i * G::WR + wr) * 64 + lane) % G::CH;
      const bool ok = row_there(key, kv, ids[i], a.c.num_pages);
      const int64_t off = row_offset(key, ids[i], a.c.page_shift, a.c.page, a.c.token) + head_off +
                          ((lin ^ swz<G>(rw)) << 4);
      uint8_t* dst = slot + (i * G::WR + wr) * 1024;
      __builtin_amdgcn_global_load_lds(ok ? (const void*)(a.c.k + off) : (const void*)g_zero, (lds_void*)dst, 16, 0, 0);
      __builtin_amdgcn_global_load_lds(ok ? (const void*)(a.c.v + off) : (const void*)g_zero,
                                       (lds_void*)(dst + G::PART), 16, 0, 0);
    }
    if constexpr (G::KV8) {
#pragma unroll
      for (int i = 0; i < G::SI; ++i) {
        const int lin = ((i * G::WR + wr) * 64) % (2 * G::TK);   // where this load's 64 scales go
        const int key = key0 + sc_key(i);
        const bool ok = row_there(key, kv, ids[G::QI + i], a.c.num_pages);
        const int64_t off = row_offset(key, ids[G::QI + i], a.c.page_shift, a.c.s_page, a.c.s_token) +
                            kvh * a.c.s_head;
        const float* src = (lin + lane >= G::TK ? a.c.v_scale : a.c.k_scale) + off;
        __builtin_amdgcn_global_load_lds(ok ? (const void*)src : (const void*)g_zero,
                                         (lds_void*)(slot + 2 * G::PART + lin * 4), 4, 0, 0);
      }
    }
  };

  acc_t o[G::DT];
#pragma unroll
  for (int d = 0; d < G::DT; ++d)
#pragma unroll
    for (int i = 0; i < AN; ++i) o[d][i] = 0.0f;
  float m = kLow, l = 0.0f;

  // ---- one stage
  auto compute = [&](int st, const uint8_t* slot) {
    const int key0 = tile_key(st);
    acc_t s[G::NKT];
#pragma unroll
    for (int kt = 0; kt < G::NKT; ++kt) {
#pragma unroll
      for (int i = 0; i < AN; ++i) s[kt][i] = 0.0f;
      const uint8_t* kr = slot + (kt * G::MT + r) * G::RB;
      const int f = swz<G>(r);   // MT is a multiple of the swizzle's period
      if constexpr (!G::KV8) {
#pragma unroll
        for (int x = 0; x < G::QS; ++x)
          s[kt] = mfma(*(const v8bf*)(kr + (((x * G::LG + g) ^ f) << 4)), q[x], s[kt]);
      } else {
#pragma unroll
        for (int x = 0; x < G::QS; x += 2) {
          const v4i u = *(const v4i*)(kr + (((x / 2 * G::LG + g) ^ f) << 4));
          s[kt] = mfma(e4m3x8_to_bf16(u[0], u[1]), q[x], s[kt]);
          s[kt] = mfma(e4m3x8_to_bf16(u[2], u[3]), q[x + 1], s[kt]);
        }
      }
    }
    const float* sc = (const float*)(slot + 2 * G::PART);
    float top = -__builtin_inff();
    const bool whole = key0 + G::TK - 1 <= p_lo && (a.window <= 0 || key0 > p_hi - a.window);
#pragma unroll
    for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
      for (int i4 = 0; i4 < AN / 4; ++i4) {
        const int kk = kt * G::MT + 8 * i4 + 4 * g;   // first of four keys
        v4f ks = {1.0f, 1.0f, 1.0f, 1.0f};
        if constexpr (G::KV8) ks = *(const v4f*)(sc + kk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[kt][4 * i4 + i];
          if constexpr (G::KV8) x *= ks[i];
          if (!whole) {
            const int j = key0 + kk + i;
            x = key_seen(j, place, a.window, a.sinks) ? x : -__builtin_inff();
          }
          s[kt][4 * i4 + i] = x;
          top = fmaxf(top, x);
        }
      }
    // scores in the exponent of 2 from here on: c s - m
    if (__any(top * c > m + kSlack)) {
      float nm = top * c;
#pragma unroll
      for (int x = G::MT; x < 64; x <<= 1) nm = fmaxf(nm, __shfl_xor(nm, x));
      nm = fmaxf(nm, m);
      const float f = __builtin_amdgcn_exp2f(m - nm);
      m = nm;
      l *= f;
#pragma unroll
      for (int d = 0; d < G::DT; ++d)
#pragma unroll
        for (int i = 0; i < AN; ++i) o[d][i] *= f;
    }
    uint32_t p[G::NKT * AN / 2];
#pragma unroll
    for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
      for (int i4 = 0; i4 < AN / 4; ++i4) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][4 * i4 + i], c, -m));
          l += e[i];
        }
        if constexpr (G::KV8) {
          const v4f vs = *(const v4f*)(sc + G::TK + kt * G::MT + 8 * i4 + 4 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] *= vs[i];
        }
        p[(kt * AN + 4 * i4) / 2] = pack_bf16(e[0], e[1]);
        p[(kt * AN + 4 * i4) / 2 + 1] = pack_bf16(e[2], e[3]);
      }
    // O^T += V^T P^T: step x takes keys kb + 4 g + {0..3} and kb + KB + 4 g + {0..3}
    constexpr int KB = G::MT == 16 ? 16 : 8;
    const int i16 = lane & 15, dh = G::MT == 32 ? ((lane >> 4) & 1) * 16 : 0;
    const uint8_t* vb = slot + G::PART;
#pragma unroll
    for (int x = 0; x < G::PS; ++x) {
      const int kb = x * G::KS;
      const v8bf pb = __builtin_bit_cast(v8bf, (v4i{(int)p[4 * x], (int)p[4 * x + 1], (int)p[4 * x + 2], (int)p[4 * x + 3]}));
#pragma unroll
      for (int d = 0; d < G::DT; ++d) {
        v8bf va;
        if constexpr (!G::KV8) {
          const int kr = 4 * g + (i16 >> 2), ch = (d * G::MT + dh) / 8 + ((i16 >> 1) & 1);
          const uint8_t* p0 = vb + (kb + kr) * G::RB + ((ch ^ swz<G>(kb + kr)) << 4) + 8 * (i16 & 1);
          const uint8_t* p1 = vb + (kb + KB + kr) * G::RB + ((ch ^ swz<G>(kb + KB + kr)) << 4) + 8 * (i16 & 1);
          const v4s a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p0);
          const v4s a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p1);
          typedef short v8s __attribute__((ext_vector_type(8)));
          va = __builtin_bit_cast(v8bf, (v8s{a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]}));
        } else {
          const int rr = i16 >> 1, kr = kb + (rr >> 2) * KB + 4 * g + (rr & 3), ch = (d * G::MT + dh) / 16;
          const uint8_t* p0 = vb + kr * G::RB + ((ch ^ swz<G>(kr)) << 4) + 8 * (i16 & 1);
          const v2i u = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)p0);
          va = e4m3x8_to_bf16((uint32_t)u[0], (uint32_t)u[1]);
        }
        o[d] = mfma(va, pb, o[d]);
      }
    }
  };

  // ---- the ring: stage st + NST - 1 goes where stage st - 1 was
  if (ns > 0) {
#pragma unroll
    for (int st = 0; st < G::NST - 1; ++st)
      if (st < ns) {
        fetch_ids(st);
        issue(st, ring + st * G::STG);
      }
    if (G::NST - 1 < ns) fetch_ids(G::NST - 1);
    int slot = 0;
    for (int st = 0; st < ns; ++st) {
      // stage st has landed once at most the later ones' loads are outstanding
      if (st + G::NST - 2 < ns) wait_vm<(G::NST - 2) * G::PW>();
      else wait_vm<0>();
      if constexpr (G::WR > 1) lds_barrier();   // ... every wave's part, and stage st - 1 is done with
      else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const int back = slot == 0 ? G::NST - 1 : slot - 1;
      if (st + G::NST - 1 < ns) {
        issue(st + G::NST - 1, ring + back * G::STG);
        if (st + G::NST < ns) fetch_ids(st + G::NST);
      }
      compute(st, ring + slot * G::STG);
      slot = slot + 1 == G::NST ? 0 : slot + 1;
    }
  }

  // ---- join the lane groups' sums and the key groups' parts, and write
#pragma unroll
  for (int x = G::MT; x < 64; x <<= 1) l += __shfl_xor(l, x);
  if constexpr (G::WK == 1) {
    const float inv = l > 0.0f ? 1.0f / l : l;             // l: 0, or NaN kept
    const float lse2 = l == 0.0f ? -__builtin_inff() : m + __builtin_amdgcn_logf(l);
    if (!live) return;
    const size_t at = (size_t)(t0 + tok) * a.heads + head;
    if (a.splits == 1) {
      uint16_t* op = a.out + at * G::D;
#pragma unroll
      for (int d = 0; d < G::DT; ++d)
#pragma unroll
        for (int i4 = 0; i4 < AN / 4; ++i4)
          *(v2i*)(op + d * G::MT + 8 * i4 + 4 * g) =
              v2i{(int)pack_bf16(o[d][4 * i4] * inv, o[d][4 * i4 + 1] * inv),
                  (int)pack_bf16(o[d][4 * i4 + 2] * inv, o[d][4 * i4 + 3] * inv)};
      if (g == 0 && a.lse) a.lse[at] = lse2 * kLn2;
    } else {
      const size_t ps = (size_t)split * a.b.tokens * a.heads + at;
      if (ns > 0) {
        float* op = a.part_o + ps * G::D;
#pragma unroll
        for (int d = 0; d < G::DT; ++d)
#pragma unroll
          for (int i4 = 0; i4 < AN / 4; ++i4)
            *(v4f*)(op + d * G::MT + 8 * i4 + 4 * g) = v4f{o[d][4 * i4] * inv, o[d][4 * i4 + 1] * inv,
                                                          o[d][4 * i4 + 2] * inv, o[d][4 * i4 + 3] * inv};
      }
      if (g == 0) a.part_lse[ps] = lse2;
    }
  } else {
    float* const so = (float*)lds;                          // [WK][ROWS][D]
    float* const sm = so + G::WK * G::ROWS * G::D;          // [2][WK][ROWS]: m, l
    __syncthreads();                                        // the ring is no longer read
    const int rl = wr * G::MT + r;
    if (g == 0) {
      sm[wk * G::ROWS + rl] = m;
      sm[(G::WK + wk) * G::ROWS + rl] = l;
    }
#pragma unroll
    for (int d = 0; d < G::DT; ++d)
#pragma unroll
      for (int i4 = 0; i4 < AN / 4; ++i4)
        *(v4f*)(so + (wk * G::ROWS + rl) * G::D + d * G::MT + 8 * i4 + 4 * g) =
            v4f{o[d][4 * i4], o[d][4 * i4 + 1], o[d][4 * i4 + 2], o[d][4 * i4 + 3]};
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
      const size_t at = (size_t)(t0 + rg / a.group) * a.heads + kvh * a.group + rg % a.group;
      if (a.splits == 1) {
        *(v2i*)(a.out + at * G::D + d) = v2i{(int)pack_bf16(ov[0] * inv, ov[1] * inv),
                                             (int)pack_bf16(ov[2] * inv, ov[3] * inv)};
        if (d == 0 && a.lse) a.lse[at] = lse2 * kLn2;
      } else {
        const size_t ps = (size_t)split * a.b.tokens * a.heads + at;
        if (ns > 0) *(v4f*)(a.part_o + ps * G::D + d) = v4f{ov[0] * inv, ov[1] * inv, ov[2] * inv, ov[3] * inv};
        if (d == 0) a.part_lse[ps] = lse2;
      }
    }
  }
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
  float mm = -__builtin_inff();
  for (int s = 0; s < a.splits; ++s) mm = fmaxf(mm, a.part_lse[s * rows + at]);
  float ll = 0.0f;
  v4f ov = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < a.splits; ++s) {
    const float x = a.part_lse[s * rows + at];
    if (x == -__builtin_inff()) continue;
    const float f = __builtin_amdgcn_exp2f(x - mm);
    const v4f y = *(const v4f*)(a.part_o + (s * rows + at) * D + d);
    ll += f;
#pragma unroll
    for (int i = 0; i < 4; ++i) ov[i] += y[i] * f;
  }
  const float inv = ll > 0.0f ? 1.0f / ll : ll;
  *(v2i*)(a.out + at * D + d) = v2i{(int)pack_bf16(ov[0] * inv, ov[1] * inv), (int)pack_bf16(ov[2] * inv, ov[3] * inv)};
  if (d == 0 && a.lse) a.lse[at] = ll == 0.0f ? -__builtin_inff() : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
}

template <class G>
hipError_t run(const AttnArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const hipError_t e = allow_lds((const void*)k_attn<G>, G::LDS, allowed);
  if (e != hipSuccess) return e;
  const int tiles = (int)(((int64_t)a.max_new * a.group + G::ROWS - 1) / G::ROWS);
  const int64_t grid = (int64_t)a.b.requests * a.c.kv_heads * a.splits * tiles;
  hipLaunchKernelGGL((k_attn<G>), dim3((unsigned)grid), dim3(G::THREADS), G::LDS, st, a);
  return hipGetLastError();
}

// The kernel for a call whose largest request has `rows` rows per kv head.
// Up to 16 and 32 rows each wave takes all of them and a part of the keys,
// without barriers; up to 64, two waves share the keys of two; beyond, four
// waves of 32 rows share every key tile.  Key groups and stages fill the LDS.
template <int D, bool KV8, class F>
auto visit_rows(int64_t rows, F f) {
  constexpr int WK = D == 256 && !KV8 ? 2 : 4;
  if (rows <= 16) return f(Geo<D, KV8, 16, 1, WK, 32, 2>{});
  if (rows <= 32) return f(Geo<D, KV8, 32, 1, WK, 32, 2>{});
  if (rows <= 64) return f(Geo<D, KV8, 32, 2, 2, 32, 2>{});
  return f(Geo<D, KV8, 32, 4, 1, D == 256 ? 32 : 64, 2>{});
}
template <class F>
auto visit(int dim, bool e4m3, int64_t rows, F f) {
  if (dim == 64) return e4m3 ? visit_rows<64, true>(rows, f) : visit_rows<64, false>(rows, f);
  if (dim == 128) return e4m3 ? visit_rows<128, true>(rows, f) : visit_rows<128, false>(rows, f);
  return e4m3 ? visit_rows<256, true>(rows, f) : visit_rows<256, false>(rows, f);
}

}  // namespace

// Enough workgroups for two on every CU, but no split shorter than four key
// tiles of the longest request: a split costs a launch and the traffic of its
// partial outputs.
int attn_splits(int, int requests, int max_new, int max_kv, int heads, int kv_heads, int dim, int e4m3, int window,
                int sinks) {
  const int64_t rows = (int64_t)max_new * (heads / kv_heads);
  int64_t keys = max_kv;
  if (window > 0 && (int64_t)window + sinks + max_new < keys) keys = (int64_t)window + sinks + max_new;
  return visit(dim, e4m3 != 0, rows, [&](auto geo) {
    typedef decltype(geo) G;
    const int64_t groups = (int64_t)requests * kv_heads * ((rows + G::ROWS - 1) / G::ROWS);
    const int64_t want = (kTargetGroups + groups - 1) / groups, most = keys / (kMinTiles * G::TT);
    const int64_t s = want < most ? want : most;
    return (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
  });
}

int launch_attn(const AttnArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  hipError_t e = visit(a.dim, a.e4m3 != 0, (int64_t)a.max_new * a.group,
                       [&](auto geo) { return run<decltype(geo)>(a, st); });
  if (e == hipSuccess && a.splits > 1) {
    const size_t rows = (size_t)a.b.tokens * a.heads, rpb = 1024 / a.dim;
    const dim3 grid((unsigned)((rows + rpb - 1) / rpb)), block(256);
    if (a.dim == 64) hipLaunchKernelGGL((k_attn_join<64>), grid, block, 0, st, a);
    else if (a.dim == 128) hipLaunchKernelGGL((k_attn_join<128>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_attn_join<256>), grid, block, 0, st, a);
    e = hipGetLastError();
  }
  return (int)e;
}

}  // namespace ocq
