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
// by direct-to-LDS loads into rings of two stages (16-byte chunks of a row
// xor-swizzled by the row, see swz), K one stage ahead of V: the products of
// the next stage run on the matrix cores while the vector unit forms the
// probabilities of this one.  V^T fragments come from LDS through the
// transposing reads.  E4M3 codes are converted exactly to bf16; the scale of a
// key multiplies its score, the scale of a value its probability.
//
// The maximum moves only when a score exceeds it by 2^8 (in the exponent of
// 2): probabilities up to 256 are as exact in bf16 and fp32 as those up to 1,
// and most tiles then need neither a cross-lane maximum nor a rescaling.
//
// Four kernels by the rows of a request (visit_rows), two ways to cut the work
// (attn_plan).  Measured on MI355X, head size 128, 32 heads on 8 kv heads, and
// what bounds each:
//   4 requests, one token over 131072 keys, bf16: 268-280 us, 6.3-6.6 TB/s of
//     the 7.1 that a streaming read reaches: HBM;
//   16 x 13 tokens over up to 4096 keys, bf16: 49-52 us, 29 of them reading at
//     the streaming rate: the piece, its ids and the first keys (5 us), loops of
//     11 to 15 stages that end between 22 and 41, writing the parts (3) and
//     joining them (5);
//   64 x 13 over up to 8192, E4M3: 175-198 us, more the longer the card has been
//     busy (HBM alone 119, products 69): conversions and softmax on the vector
//     unit, matrix cores 32 % busy;
//   NVFP4 (codes converted to fp16 by every wave, an instruction and a half a pair of
//     values with the scale): 4 requests, one token over 131072 keys 94-96 us, 5.2
//     TB/s (HBM, and 18 us around the loops: pieces, parts, join); 16 x 13 over 4096
//     41-44, 64 x 13 over 8192 170-180 (vector unit 57 %, matrix cores 25 % busy);
//   2048 new tokens over 10007 keys, bf16: 898-953 TFLOP/s (8192 over 12288:
//     951-1020; a library product of 8192^3: 1202): vector unit and matrix cores
//     together, 45 % of the matrix cores' cycles.
#include "gemm_core.h"
#include "layer_dev.h"
#include "layer_index.h"

#include <type_traits>

namespace ocq {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v2i lds_v2i;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLow = -3.4028234663852886e38f;   // below every score that is visible
constexpr float kSlack = 8.0f;                    // see above
// NVFP4, widened or not: probabilities are fp16, up to 2^(8 + 7) of its 65504, so that only those
// below 2^-31 of the largest round as if they were 0
constexpr float kUp = 7.0f;

constexpr int kTargetGroups = 512, kMinTiles = 4, kMaxSplits = 256;   // see attn_plan
constexpr int kEvenRequests = 256;                // requests of a batch that is cut into pieces

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

constexpr int LG_(int MT) { return 64 / MT; }
template <int MT> struct Acc;
template <> struct Acc<16> { typedef v4f T; };
template <> struct Acc<32> { typedef v16f T; };

__device__ __forceinline__ v4f mfma(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v16f mfma(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma(v8h a, v8h b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v16f mfma(v8h a, v8h b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// D: head size; KV8: E4M3 cache; MT: rows of a wave; WR x
// WK waves: over the rows and over the keys; TK: keys of a wave's stage; MINW:
// waves per SIMD that the registers leave room for.  NST: slots of each ring;
// two, so that the loop over the stages, unrolled by two, has every LDS address
// as a register that does not change plus a constant.
template <int D_, int FMT_, int MT_, int WR_, int WK_, int TK_, int MINW_>
struct Geo {
  static constexpr int MINW = MINW_, NST = 2;
  static constexpr int D = D_, MT = MT_, WR = WR_, WK = WK_, TK = TK_;
  static constexpr bool KV8 = FMT_ == OCQ_CACHE_E4M3, KV4 = FMT_ == OCQ_CACHE_NVFP4;
  static constexpr bool WIDE = FMT_ == kWidened;                        // only keys below wide_keys are there
  static constexpr bool F16 = KV4 || WIDE;                              // operands of the products: fp16, or bf16
  static constexpr int NW = WR * WK, THREADS = 64 * NW, ROWS = MT * WR;
  static constexpr int RB = KV4 ? D / 2 : KV8 ? D : 2 * D, CH = RB / 16;   // bytes and chunks of a row
  static constexpr int PART = TK * RB;                                  // K (or V) bytes of a key group's stage
  static constexpr int SB = KV4 ? D / 16 : 4;                           // bytes of a key's scales
  static constexpr int SCB = KV4 ? (TK * SB > 256 ? TK * SB : 256) : KV8 ? 256 : 0;   // the stage's
  static constexpr int KSTG = PART + SCB + 256, VSTG = PART + SCB;      // a stage of K (with 64 page ids) and of V
  static constexpr int VTAB = KV4 ? TK * SB * 2 : 0;                    // a wave's fp16 scales of V, key by key
  static constexpr int RING = WK * NST * (KSTG + VSTG);
  static constexpr int QI = (PART / 1024 + WR - 1) / WR;                // K (or V) loads per wave and stage
  static constexpr int SL = KV4 ? SCB / 256 : 1;                        // loads of its scales, and a wave's of them
  static constexpr int SI = KV4 ? (SL + WR - 1) / WR : KV8 ? 1 : 0;
  static constexpr int PW = 2 * QI + 1 + 2 * SI;                        // all loads per wave and stage
  static constexpr int KW = KV4 ? (RB / LG_(MT) >= 16 ? 4 : 2) : KV8 ? 2 : 1;   // steps of S that a read of K serves
  static constexpr int AHEAD = WR > 1 ? NST - 1 : NST;                  // stages on their way, see the ring
  static constexpr int TT = TK * WK;                                    // keys of a tile, all key groups
  static constexpr int NKT = TK / MT;                                   // key tiles of a stage
  static constexpr int KS = 512 / MT;                                   // inputs of one MFMA (32 or 16)
  static constexpr int QS = D / KS, DT = D / MT, LG = 64 / MT;          // steps of S, tiles of O, lane groups
  static constexpr int PS = TK / KS;                                    // steps of O
  static constexpr int SO = D + 4;                                      // floats of a joined row: 16 bytes further per row
  static constexpr int JOIN = WK > 1 ? WK * ROWS * (SO * 4 + 8) + 4 : 0;
  static constexpr int LDS = RING + NW * VTAB > JOIN ? RING + NW * VTAB : JOIN;
  static constexpr bool EVEN = WK > 1;                                  // may be cut into pieces (layer_index.h)
  // Tiles of the smallest piece.  A stage of 4-bit keys takes a wave alone as long as
  // its loads (2.3 us): two tiles (4 requests, one token over 1100 / 2200 / 4400 / 8800
  // keys 14.2, 14.6, 19.9, 24.3 us; four tiles 16.4, 16.6, 18.7, 26.2).  For more rows
  // four as well (16 x 13 over 1000 keys 22.7; two tiles 26.9).
  static constexpr int MIN_TILES = KV4 && MT == 16 ? 2 : kMinTiles;
  static constexpr int PER_CU = 160 * 1024 / (LDS + 1024) < 4 * MINW / NW ? 160 * 1024 / (LDS + 1024) : 4 * MINW / NW;
  static constexpr int RESIDENT = 256 * (PER_CU > 0 ? PER_CU : 1);      // workgroups at once, 256 CUs
  static_assert(PART % 1024 == 0 && (PART % (1024 * WR) == 0 || KV4) && TK % 32 == 0 && LDS <= 160 * 1024, "");
  static_assert(TK <= 64, "one load for the ids, and for the scales");
  static_assert(!KV4 || TK == 64 || (MT == 32 && TK == 32), "a transposing read of codes takes 64 or 32 keys");
};

// Chunk swizzle: chunk c of row `row` lies at chunk c ^ swz(row).  What one
// pass of the banks (256 bytes) takes has to lie in different banks:
//   K   16 rows (16-byte reads), one chunk of each: swz takes 16 values over
//       16 rows, or 16 RB / 256 where a pass holds several rows;
//   V   half a wave's transposing reads: for bf16 4 rows x 4 chunks (MT 32) or
//       8 rows x 2 chunks (MT 16) from row 0 or 4 g, for codes 4 + 4 rows KB
//       apart x 2 chunks, or 8 + 8 rows x 1 chunk; for NVFP4 16 rows x 1 chunk
//       (MT 32), or 32 rows x half a chunk, which takes two passes at least.
// So the row bits of V's pass go to the chunk bits above those it reads
// together.  Linear in the bits (swz(a + b) = swz(a) ^ swz(b) without carries).
template <class G>
__device__ __forceinline__ constexpr int swz(int row) {
  const int b0 = row & 1, b1 = row >> 1 & 1, b2 = row >> 2 & 1, b3 = row >> 3 & 1, b4 = row >> 4 & 1;
  if constexpr (G::KV4) {
    const int b5 = row >> 5 & 1;
    if constexpr (G::MT == 32)
      return G::CH == 8 ? b1 | b3 << 1 | (b2 ^ b4) << 2 : G::CH == 4 ? (b2 ^ b4) | b3 << 1 : b3;
    else
      return G::CH == 8 ? b1 | (b2 ^ b4) << 1 | (b3 ^ b5) << 2 : G::CH == 4 ? (b2 ^ b4) | (b3 ^ b5) << 1 : b3 ^ b4;
  } else if constexpr (!G::KV8) {
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

// 16 (or 4) bytes from p for each lane to LDS, lane after lane from `to`.  The
// address is a chosen one, not a branch to one of two loads.
// ONCE: nobody else reads these bytes (non-temporal: they pass through L2
// without staying; 4 x 131072 keys: 314 -> 280 us).
template <bool ONCE>
__device__ __forceinline__ void dma16(uint64_t p, uint8_t* to) {
  asm("" : "+v"(p));
  if constexpr (ONCE) __builtin_amdgcn_global_load_lds((const void*)p, (lds_void*)to, 16, 0, 2);
  else __builtin_amdgcn_global_load_lds((const void*)p, (lds_void*)to, 16, 0, 0);
}
__device__ __forceinline__ void dma4(uint64_t p, uint8_t* to) {
  asm("" : "+v"(p));
  __builtin_amdgcn_global_load_lds((const void*)p, (lds_void*)to, 4, 0, 0);
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

// The same of 4-bit codes: 16 keys of one d per lane each.
template <int O0, int O1, int O2, int O3>
__device__ __forceinline__ void read_tr4(v2i (&x)[4], const uint32_t (&ad)[4]) {
  asm volatile(
      "ds_read_b64_tr_b4 %0, %4 offset:%8\n\tds_read_b64_tr_b4 %1, %5 offset:%9\n\t"
      "ds_read_b64_tr_b4 %2, %6 offset:%10\n\tds_read_b64_tr_b4 %3, %7 offset:%11\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
      : "v"(ad[0]), "v"(ad[1]), "v"(ad[2]), "v"(ad[3]), "n"(O0), "n"(O1), "n"(O2), "n"(O3));
}

// eight E2M1 codes (low nibble first) times their own scales in pairs -> fp16, exact
__device__ __forceinline__ v8h e2m1x8_pairs(uint32_t d, const v2h* s) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 0) * s[0];
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 1) * s[1];
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 2) * s[2];
  const v2h e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 3) * s[3];
  return v8h{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {   // nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2h));
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
  return G::KW * (G::KS * (s / G::KW) + 8 * g) + 8 * (s % G::KW);   // one read of K serves KW steps
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

// The request that a workgroup belongs to.
struct Found {
  int req, t0, n, kv;   // request (-1: none), its first new token, their number, its cached tokens
  int tiles, pieces;    // of each of its segments
  int first;            // its first piece (kv head 0)
};

// Every wave cuts the batch into pieces by itself, in registers: lane l holds
// request base + l.
__device__ __forceinline__ Found find_piece(const AttnArgs& a, int TT, int min_tiles, int piece) {
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
  int id = lane;   // the request that a lane holds (less its base)
  float per;
  if (2 * segments > a.slots) {
    // about as many segments as slots, or more: only those of one and a half
    // mean shares and more are cut (pieces of half a share: 64 x 13 rows over
    // 8192 keys in E4M3 221 us instead of 203)
    per = (float)(total / 2 * 3 / a.slots + 1);
    if (a.format != OCQ_CACHE_BF16 && a.b.requests <= 64) {
      // The longest first, so that a CU's second workgroup is a short one: E4M3
      // keys are bound by the CUs' vector units (64 x 13 rows over 8192: 189 ->
      // 181 us), bf16 keys by HBM (40 x 13 rows over 4096: 99 -> 102).
      int rank = 0;
      for (int r = 0; r < a.b.requests; ++r) {
        const int other = __builtin_amdgcn_readlane(T, r);
        rank += other > T || (other == T && r < lane);
      }
      rank = lane < a.b.requests ? 4 * rank : 4 * lane;
      T = __builtin_amdgcn_ds_permute(rank, T);
      t0 = __builtin_amdgcn_ds_permute(rank, t0);
      n = __builtin_amdgcn_ds_permute(rank, n);
      kv = __builtin_amdgcn_ds_permute(rank, kv);
      id = __builtin_amdgcn_ds_permute(rank, id);
    }
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
  per = fmaxf(per, (float)min_tiles);
  const float inv = 1.0f / per;
  Found f{-1, 0, 0, 0, 0, 0, 0};
  int carry = 0;
  for (int base = 0; base < a.b.requests; base += 64) {
    if (base > 0) T = load(base, t0, n, kv);
    const int c = piece_count(T, inv), end = wave_scan(c * kvh) + carry;
    // the lane whose request it is
    const uint64_t who = __ballot(piece < end && piece >= end - c * kvh);
    if (who) {
      const int l = __builtin_ctzll(who);
      f.req = base + __builtin_amdgcn_readlane(id, l);
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
  int pieces, index;    // of the segment, and which one this is
};

// Joins N rows' parts: ov[k] = sum_i 2^(lse_i - mm) out_i and ll[k] = sum_i
// 2^(lse_i - mm) over the `parts` parts of row k (part i at row_of(i, k)), mm[k]
// the largest lse; a part without keys (lse -inf) has no output.  B parts of
// every row are read at a time.  SHARED: other workgroups of the same launch
// wrote the parts, which lie past the L2 of one XCD (see put_part).
template <bool SHARED, int N, int B, class F>
__device__ __forceinline__ void join_parts(const AttnArgs& a, int parts, const int (&d)[N], int D, F row_of,
                                           float (&mm)[N], float (&ll)[N], v4f (&ov)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    mm[k] = -__builtin_inff();
    ll[k] = 0.0f;
    ov[k] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  for (int i0 = 0; i0 < parts; i0 += B) {
    float x[N][B];
    v4f y[N][B];
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const size_t r = row_of(i0 + j < parts ? i0 + j : parts - 1, k);
        if constexpr (SHARED) {
          x[k][j] = __hip_atomic_load(a.part_lse + r, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          const uint64_t* p = (const uint64_t*)(a.part_o + r * D + d[k]);
          const uint64_t lo = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          const uint64_t hi = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          const v2f a0 = __builtin_bit_cast(v2f, lo), a1 = __builtin_bit_cast(v2f, hi);
          y[k][j] = v4f{a0[0], a0[1], a1[0], a1[1]};
        } else {
          x[k][j] = a.part_lse[r];
          y[k][j] = *(const v4f*)(a.part_o + r * D + d[k]);
        }
      }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float nm = mm[k];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (i0 + j >= parts) x[k][j] = -__builtin_inff();
        nm = fmaxf(nm, x[k][j]);
      }
      const bool none = nm == -__builtin_inff();   // nothing yet (NaN goes on)
      const float f = none ? 1.0f : __builtin_amdgcn_exp2f(mm[k] - nm);
      ll[k] *= f;
#pragma unroll
      for (int i = 0; i < 4; ++i) ov[k][i] *= f;
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const float e = x[k][j] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(x[k][j] - nm);
        ll[k] += e;
#pragma unroll
        for (int i = 0; i < 4; ++i) ov[k][i] += x[k][j] == -__builtin_inff() ? 0.0f : y[k][j][i] * e;
      }
      mm[k] = nm;
    }
  }
}

// A joined row's four values and its lse.
__device__ __forceinline__ void put_joined(const AttnArgs& a, size_t at, int d, int D, v4f ov, float mm, float ll) {
  const float inv = ll > 0.0f ? 1.0f / ll : ll;
  *(v2i*)(a.out + at * D + d) = v2i{(int)pack_bf16(ov[0] * inv, ov[1] * inv), (int)pack_bf16(ov[2] * inv, ov[3] * inv)};
  if (d == 0 && a.lse) a.lse[at] = ll == 0.0f ? -__builtin_inff() : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
}

// A part's four values (and its lse with d = 0), for a workgroup on any XCD to
// read in the same launch: device-scope stores (sc1) write through the XCD's
// L2.  They are visible to device-scope loads once the wave's count of
// outstanding stores is 0.  The wait state keeps the compiler's next instruction
// from overwriting the data as the store reads it (it inserts one itself after
// stores of more than 8 bytes that it can see).
__device__ __forceinline__ void put_part(const AttnArgs& a, size_t row, int d, int D, v4f y, float lse2) {
  asm volatile("global_store_dwordx4 %0, %1, off sc1\n\ts_nop 0" ::"v"(a.part_o + row * D + d), "v"(y) : "memory");
  if (d == 0) __hip_atomic_store(a.part_lse + row, lse2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The last key that rows up to place p_hi can see.
template <class G>
__device__ __forceinline__ int last_key(const AttnArgs& a, int p_hi) {
  return G::WIDE && p_hi >= a.wide_keys ? a.wide_keys - 1 : p_hi;
}

template <class G>
__device__ __forceinline__ void attend(const AttnArgs& a, const Piece& pc, uint8_t* lds) {
  typedef typename Acc<G::MT>::T acc_t;
  constexpr int AN = G::MT == 16 ? 4 : 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave % G::WR, wk = wave / G::WR;
  const int r = lane % G::MT, g = lane / G::MT;
  const int n = pc.n, t0 = pc.t0, kv = pc.kv, base = pc.base, row0 = pc.row0, kvh = pc.kvh;
  const int p_lo = pc.p_lo, p_hi = pc.p_hi, ns = pc.s1 - pc.s0;

  // this lane's row: in the tile, of the request, of the output
  const int rl = wr * G::MT + r, row = row0 + rl;
  const bool live = row < n * a.group;
  const int tok = live ? row / a.group : 0, head = kvh * a.group + (live ? row % a.group : 0);
  const int place = live ? base + tok : -1;
  const size_t at = (size_t)(t0 + tok) * a.heads + head;
  typedef std::conditional_t<G::F16, v8h, v8bf> operand;
  operand q[G::QS];
  const uint16_t* qp = a.q + (t0 + tok) * a.q_token + head * a.q_head;
  float c = a.scale * kLog2e;
  v4i q_bits[G::QS];
#pragma unroll
  for (int s = 0; s < G::QS; ++s) {
    q_bits[s] = live ? *(const v4i*)(qp + q_dim<G>(s, g)) : v4i{0, 0, 0, 0};
    if constexpr (!G::F16) q[s] = __builtin_bit_cast(operand, q_bits[s]);
  }
  // Codes times their scales are exact in fp16, not all in bf16 with one
  // instruction less; q goes to fp16 after a power of two that brings the row's
  // largest value to 2^14 .. 2^15, which is exact down to 2^-28 of it (and off by
  // at most 2^-39 of it below).  The factor c takes the power back, and k's unit, in
  // one step: c times the unit alone may be past 32 bits where the product is not.
  // It stays a normal number: a masked score is -inf, and 0 times it is none, nor is
  // inf times a score of 0.  (Scores are below 2^36 here: a c of less than 2^-126
  // makes them all 0 beside any other one, 2^-126 too.)  (Called while the first
  // page ids are on their way.)
  auto q_to_f16 = [&](auto& to) {
    float f[G::QS][8], top = 0.0f;
#pragma unroll
    for (int s = 0; s < G::QS; ++s) {
      unpack8_bf16(q_bits[s], f[s]);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[s][j]));
    }
#pragma unroll
    for (int x = G::MT; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    const int up = top > 0.0f && top < __builtin_inff() ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
    for (int s = 0; s < G::QS; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) to[s][j] = (_Float16)__builtin_ldexpf(f[s][j], up);
    c = __builtin_ldexpf(c, __builtin_amdgcn_frexp_expf(a.c.k_unit) - 1 - up);
    c = __builtin_amdgcn_fmed3f(c, 0x1p-126f, 0x1.fffffep127f);
  };

  // ---- loads: rows of this wave's part of its key group's stage.  V of a stage
  // goes after K of it, with the same offsets.
  uint8_t* const ring = lds + wk * G::RING / G::WK;
  auto k_slot = [](int i) constexpr { return i * G::KSTG; };                       // offsets in the ring
  auto v_slot = [](int i) constexpr { return G::NST * G::KSTG + i * G::VSTG; };
  const int32_t* const table = a.b.table + pc.req * a.b.table_stride;
  const int page_mask = (1 << a.c.page_shift) - 1;
  const uint64_t k_head = (uint64_t)a.c.k + kvh * a.c.head, v_less_k = (uint64_t)a.c.v - (uint64_t)a.c.k;
  constexpr int SE = G::KV4 ? 1 : 4;                     // bytes that strides of the scales count
  const uint64_t ks_head = (uint64_t)a.c.k_scale + (G::SI ? kvh * a.c.s_head * SE : 0);
  const uint64_t vs_less_ks = (uint64_t)a.c.v_scale - (uint64_t)a.c.k_scale;
  // first key of the wave's key group in stage st: a multiple of TK, so that a
  // row's place in its page is that of the first key plus a part of its own
  auto tile_key = [&](int st) { return tile_of(pc.tiles, pc.s0 + st) * G::TT + wk * G::TK; };
  // load i of the stage's PART / 1024 (where waves outnumber them, some come twice)
  auto nth = [&](int i) { return (i * G::WR + wr) % (G::PART / 1024); };
  auto s_nth = [&](int i) { return G::SL == 1 ? 0 : (i * G::WR + wr) % G::SL; };
  auto q_row = [&](int i) {   // row of load i of K and V, or (from i = QI) of the scales
    if (i < G::QI) return (nth(i) * 64 + lane) / G::CH;
    return G::KV4 ? (s_nth(i - G::QI) * 64 + lane) / (G::SB / 4) % G::TK : lane % G::TK;
  };
  uint32_t part[G::QI], s_part[G::SI + 1];
#pragma unroll
  for (int i = 0; i < G::QI; ++i) {
    const int rw = q_row(i), lin = (nth(i) * 64 + lane) % G::CH;
    part[i] = (rw & page_mask) * a.c.token + ((lin ^ swz<G>(rw)) << 4);
  }
#pragma unroll
  for (int i = 0; i < G::SI; ++i)
    s_part[i] = (q_row(G::QI + i) & page_mask) * a.c.s_token * SE + (G::KV4 ? lane % (G::SB / 4) * 4 : 0);
  const uint64_t zero = (uint64_t)g_zero;
  const KeyRange range = key_range(p_lo, last_key<G>(a, p_hi), a.window, a.sinks);
  uint64_t src[G::QI], s_src[G::SI + 1];   // rows of the last K stage issued
  bool there[G::QI], s_there[G::SI + 1];
  // Page ids come with the K stage AHEAD before the one that they are for: a
  // load into registers would have to be waited for together with every
  // earlier load of the wave.
  auto entry = [&](int st, int row) { return table + table_entry(tile_key(st) + row, kv, a.c.page_shift); };
  auto issue_k = [&](int st, int slot, auto id_of) {
    const int key0 = tile_key(st);
    int ids[G::QI], sid[G::SI + 1];
#pragma unroll
    for (int i = 0; i < G::QI; ++i) ids[i] = id_of(i);
#pragma unroll
    for (int i = 0; i < G::SI; ++i) sid[i] = id_of(G::QI + i);
    if constexpr (G::WR == 1) {
      // The next ids go where these lay: they have to be read, not only asked
      // for, before (waves that share a stage read them from the other slot).
#pragma unroll
      for (int i = 0; i < G::QI; ++i) asm volatile("" : "+v"(ids[i]) : : "memory");
#pragma unroll
      for (int i = 0; i < G::SI; ++i) asm volatile("" : "+v"(sid[i]) : : "memory");
    }
    uint8_t* const to = ring + slot;
    dma4((uint64_t)entry(st + G::AHEAD < ns ? st + G::AHEAD : st, lane % G::TK), to + G::PART + G::SCB);
    const uint64_t first = k_head + (uint32_t)(key0 & page_mask) * a.c.token;
#pragma unroll
    for (int i = 0; i < G::QI; ++i) there[i] = page_there(ids[i], a.c.num_pages);
#pragma unroll
    for (int i = 0; i < G::SI; ++i) s_there[i] = page_there(sid[i], a.c.num_pages);
    if (key0 + G::TK - 1 > range.to || key0 <= range.from) {   // a stage at the edge of what the rows see
      asm volatile("");
#pragma unroll
      for (int i = 0; i < G::QI; ++i) there[i] = there[i] && key_in(key0 + q_row(i), range);
#pragma unroll
      for (int i = 0; i < G::SI; ++i) s_there[i] = s_there[i] && key_in(key0 + q_row(G::QI + i), range);
    }
#pragma unroll
    for (int i = 0; i < G::QI; ++i) {
      src[i] = first + (uint64_t)(uint32_t)ids[i] * a.c.page + part[i];
      dma16<G::EVEN>(there[i] ? src[i] : zero, to + nth(i) * 1024);
    }
#pragma unroll
    for (int i = 0; i < G::SI; ++i) {
      s_src[i] = ks_head + (uint64_t)(uint32_t)(key0 & page_mask) * a.c.s_token * SE +
                 (uint64_t)(uint32_t)sid[i] * a.c.s_page * SE + s_part[i];
      dma4(s_there[i] ? s_src[i] : zero, to + G::PART + s_nth(i) * 256);
    }
  };
  auto issue_v = [&](int slot) {
    uint8_t* const to = ring + slot;
#pragma unroll
    for (int i = 0; i < G::QI; ++i) dma16<G::EVEN>(there[i] ? src[i] + v_less_k : zero, to + nth(i) * 1024);
#pragma unroll
    for (int i = 0; i < G::SI; ++i) dma4(s_there[i] ? s_src[i] + vs_less_ks : zero, to + G::PART + s_nth(i) * 256);
  };

  acc_t o[G::DT];
  float m = kLow, l = 0.0f;
#pragma unroll
  for (int d = 0; d < G::DT; ++d)
#pragma unroll
    for (int i = 0; i < AN; ++i) o[d][i] = 0.0f;

  // where the lane's part of a V^T fragment lies in a stage: tile d of the
  // output, keys kb + 4 g + {0..3} (first half) and kb + KB + 4 g + {0..3}
  uint32_t v_off[G::DT][G::KV8 || G::KV4 ? 1 : 2];
  {
    constexpr int KB = G::MT == 16 ? 16 : 8;
    const int i16 = lane & 15, dh = G::MT == 32 ? ((lane >> 4) & 1) * 16 : 0;
#pragma unroll
    for (int d = 0; d < G::DT; ++d)
#pragma unroll
      for (int h = 0; h < (G::KV8 || G::KV4 ? 1 : 2); ++h) {
        if constexpr (G::KV4) {   // codes: a lane names the 16 of one key, keys KB apart four at a time
          const int key = (i16 >> 2) * KB + 4 * g + (i16 & 3), blk = (d * G::MT + dh) / 16;
          v_off[d][h] = (uint32_t)(uintptr_t)(lds_void*)ring + key * G::RB + (((blk >> 1) ^ swz<G>(key)) << 4) + 8 * (blk & 1);
          continue;
        }
        const int key = G::KV8 ? (i16 >> 3) * KB + 4 * g + ((i16 >> 1) & 3) : h * KB + 4 * g + (i16 >> 2);
        const int ch = G::KV8 ? (d * G::MT + dh) / 16 : (d * G::MT + dh) / 8 + ((i16 >> 1) & 1);
        v_off[d][h] = (uint32_t)(uintptr_t)(lds_void*)ring + key * G::RB + ((ch ^ swz<G>(key)) << 4) + 8 * (i16 & 1);
      }
  }

  // ---- one stage: S^T = K Q^T
  typedef acc_t scores[G::NKT];
  uint32_t k_off[G::QS / G::KW];   // the lane's part of the K fragments, key tile 0
#pragma unroll
  for (int x = 0; x < G::QS / G::KW; ++x) {
    if constexpr (G::KV4 && G::KW == 2)
      k_off[x] = r * G::RB + ((((x * G::LG + g) >> 1) ^ swz<G>(r)) << 4) + 8 * (g & 1);
    else
      k_off[x] = r * G::RB + (((x * G::LG + g) ^ swz<G>(r)) << 4);
  }
  auto products = [&](auto slot_c, scores& s) {
    constexpr int slot = decltype(slot_c)::value;
    // codes and scales of the whole stage before the first product: the compiler
    // would ask for them one by one and wait for each
    constexpr int NX = G::KV4 ? G::QS / G::KW : 1;
    typedef std::conditional_t<G::KW == 4, v4i, v2i> codes_t;
    codes_t k_raw[G::NKT][NX];
    uint32_t k_sc[G::NKT][NX];
    if constexpr (G::KV4) {
#pragma unroll
      for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          const uint8_t* const sc = ring + slot + G::PART + (kt * G::MT + r) * G::SB + (x * G::LG + g) * (G::KW / 2);
          k_sc[kt][x] = G::KW == 4 ? *(const uint16_t*)sc : *sc;
          k_raw[kt][x] = *(const codes_t*)(ring + slot + kt * G::MT * G::RB + (k_off[x] ^ (swz<G>(kt * G::MT) << 4)));
        }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int kt = 0; kt < G::NKT; ++kt) {
#pragma unroll
      for (int i = 0; i < AN; ++i) s[kt][i] = 0.0f;
      // (swz of the tile's first row is not 0 in the E4M3 layouts of 16-row tiles)
      const int at = slot + kt * G::MT * G::RB, f = swz<G>(kt * G::MT) << 4;
      if constexpr (G::KV4) {
#pragma unroll
        for (int x = 0; x < G::QS; x += G::KW) {
          v2h s0, s1;
          e4m3x2_scales(k_sc[kt][x / G::KW], s0, s1);
#pragma unroll
          for (int j = 0; j < G::KW; ++j)
            s[kt] = mfma(e2m1x8_to_f16((uint32_t)k_raw[kt][x / G::KW][j], j < 2 ? s0 : s1), q[x + j], s[kt]);
        }
      } else if constexpr (!G::KV8) {
#pragma unroll
        for (int x = 0; x < G::QS; ++x) {
          const operand ka = *(const operand*)(ring + at + (k_off[x] ^ f));
          s[kt] = mfma(ka, q[x], s[kt]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < G::QS; x += 2) {
          const v4i u = *(const v4i*)(ring + at + (k_off[x / 2] ^ f));
          const v8bf k0 = e4m3x8_to_bf16(u[0], u[1]), k1 = e4m3x8_to_bf16(u[2], u[3]);
          s[kt] = mfma(k0, q[x], s[kt]);
          s[kt] = mfma(k1, q[x + 1], s[kt]);
        }
      }
    }
  };
  // the keys' scales and the mask
  auto finish = [&](int st, auto slot_c, scores& s) {
    const int key0 = tile_key(st);
    const float* sc = (const float*)(ring + decltype(slot_c)::value + G::PART);
    if constexpr (G::KV8) {
#pragma unroll
      for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
        for (int i4 = 0; i4 < AN / 4; ++i4) {
          const v4f ks = *(const v4f*)(sc + kt * G::MT + 8 * i4 + 4 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[kt][4 * i4 + i] *= ks[i];
        }
    }
    if (key0 + G::TK - 1 > p_lo || (a.window > 0 && key0 <= p_hi - a.window) || (G::WIDE && key0 + G::TK > a.wide_keys)) {
      asm volatile("");   // a branch, not selects in every stage
#pragma unroll
      for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
        for (int i = 0; i < AN; ++i) {
          const int j = key0 + kt * G::MT + 8 * (i >> 2) + 4 * g + (i & 3);
          const bool seen = key_seen(j, place, a.window, a.sinks) && (!G::WIDE || j < a.wide_keys);
          s[kt][i] = seen ? s[kt][i] : -__builtin_inff();
        }
    }
  };
  // Stage st from its scores sa: the maximum, then the probabilities while the
  // products of the next stage (into sb) run on the matrix cores, then O.
  auto step = [&](auto k_next, auto v_at, scores& sa, scores& sb) {
    float top = -__builtin_inff();
#pragma unroll
    for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
      for (int i = 0; i < AN; ++i) top = fmaxf(top, sa[kt][i]);
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
    _Float16* const v_tab = (_Float16*)(lds + G::RING + wave * G::VTAB);   // [D / 16][TK]
    if constexpr (G::KV4) {
      // the stage's scales of V in fp16, so that a lane finds those of four keys
      // side by side: its part of a V^T fragment has a scale for every key
      constexpr int HALF = G::TK == 64 ? G::SB : G::SB / 2;                // scales of a key that one lane takes
      const uint8_t* const from = ring + decltype(v_at)::value + G::PART + lane % G::TK * G::SB + lane / G::TK * HALF;
#pragma unroll
      for (int j = 0; j < HALF; j += 2) {
        const v2h two = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)*(const uint16_t*)(from + j), 1.0f, false);
        v_tab[(lane / G::TK * HALF + j) * G::TK + lane % G::TK] = two[0];
        v_tab[(lane / G::TK * HALF + j + 1) * G::TK + lane % G::TK] = two[1];
      }
    }
    products(k_next, sb);
    const float* sc = (const float*)(ring + decltype(v_at)::value + G::PART);
    const float from = G::F16 ? kUp - m : -m;
    uint32_t p[G::NKT * AN / 2];
#pragma unroll
    for (int kt = 0; kt < G::NKT; ++kt)
#pragma unroll
      for (int i4 = 0; i4 < AN / 4; ++i4) {
        v4f vs = {1.0f, 1.0f, 1.0f, 1.0f};
        if constexpr (G::KV8) vs = *(const v4f*)(sc + kt * G::MT + 8 * i4 + 4 * g);
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sa[kt][4 * i4 + i], c, from));
          l += e[i];
          if constexpr (G::KV8) e[i] *= vs[i];
        }
        // bf16 is what the matrix instruction takes beside bf16 (or converted)
        // values: an output is off by 0.0023 of its size where its own rounding
        // is 0.0017.  Two halves of each probability would double the products.
        p[(kt * AN + 4 * i4) / 2] = G::F16 ? pack_f16(e[0], e[1]) : pack_bf16(e[0], e[1]);
        p[(kt * AN + 4 * i4) / 2 + 1] = G::F16 ? pack_f16(e[2], e[3]) : pack_bf16(e[2], e[3]);
      }
    if constexpr (G::KV4) {
      // Fragment f: keys of steps 2 y and 2 y + 1, tile d of the output, f = y DT + d.
      // Codes of four fragments at a time, scales of the next fragment while this one
      // is multiplied (the compiler would ask for them when they are needed).
      constexpr int NF = G::PS / 2 * G::DT, KB = G::MT == 16 ? 16 : 8;
      const int dh = G::MT == 32 ? (lane >> 4) & 1 : 0;
      const _Float16* const v_sc = v_tab + dh * G::TK + 4 * g;
      v4h vs[2][4];   // the scales of the lane's 16 keys, of this fragment and the next
      auto scales_of = [&](int f, v4h (&to)[4]) {
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
          to[k4] = *(const v4h*)(v_sc + f % G::DT * (G::MT / 16) * G::TK + f / G::DT * 2 * G::KS + k4 * KB);
      };
      scales_of(0, vs[0]);
      unrolled<NF / 4>([&](auto blk) {
        constexpr int F0 = 4 * decltype(blk)::value;
        auto at_key = [](int f) constexpr { return decltype(v_at)::value + f / G::DT * 2 * G::KS * G::RB; };
        uint32_t ad[4];
        v2i x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) ad[j] = v_off[(F0 + j) % G::DT][0];
        read_tr4<at_key(F0), at_key(F0 + 1), at_key(F0 + 2), at_key(F0 + 3)>(x, ad);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int f = F0 + j, y = f / G::DT, d = f % G::DT;
          if (f + 1 < NF) scales_of(f + 1, vs[(f + 1) & 1]);
          __builtin_amdgcn_sched_barrier(0);
          const v4h(&sc)[4] = vs[f & 1];
          v2h pair[8];
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            pair[2 * k4] = __builtin_shufflevector(sc[k4], sc[k4], 0, 1);
            pair[2 * k4 + 1] = __builtin_shufflevector(sc[k4], sc[k4], 2, 3);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int st2 = 2 * y + h;
            const v8h pb = __builtin_bit_cast(
                v8h, (v4i{(int)p[4 * st2], (int)p[4 * st2 + 1], (int)p[4 * st2 + 2], (int)p[4 * st2 + 3]}));
            o[d] = mfma(e2m1x8_pairs((uint32_t)x[j][h], pair + 4 * h), pb, o[d]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      });
      return;
    }
    // O^T += V^T P^T, four fragments (step x of the keys, tile d of the output) at a time
    if constexpr (!G::KV4) unrolled<G::PS * G::DT / 4>([&](auto blk) {
      constexpr int F0 = 4 * decltype(blk)::value;
      auto at_key = [](int f) constexpr { return decltype(v_at)::value + f / G::DT * G::KS * G::RB; };
      operand va[4];
      if constexpr (!G::KV8) {
        uint32_t ad[8];
        v2i x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) ad[j] = v_off[(F0 + j / 2) % G::DT][j & 1];
        read_tr16<at_key(F0), at_key(F0 + 1), at_key(F0 + 2), at_key(F0 + 3)>(x, ad);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          va[j] = __builtin_bit_cast(operand, __builtin_shufflevector(x[2 * j], x[2 * j + 1], 0, 1, 2, 3));
      } else {
        uint32_t ad[4];
        v2i x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) ad[j] = v_off[(F0 + j) % G::DT][0];
        read_tr8<at_key(F0), at_key(F0 + 1), at_key(F0 + 2), at_key(F0 + 3)>(x, ad);
#pragma unroll
        for (int j = 0; j < 4; ++j) va[j] = e4m3x8_to_bf16((uint32_t)x[j][0], (uint32_t)x[j][1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        constexpr int DT = G::DT;
        const int x = (F0 + j) / DT, d = (F0 + j) % DT;
        const operand pb = __builtin_bit_cast(
            operand, (v4i{(int)p[4 * x], (int)p[4 * x + 1], (int)p[4 * x + 2], (int)p[4 * x + 3]}));
        o[d] = mfma(va[j], pb, o[d]);
      }
    });
  };

  // ---- the rings.  Iteration st takes V of stage st and K of stage st + 1 (the
  // last one multiplies a K that nobody uses).  Waves that share a stage meet
  // once per iteration: then its loads have landed, K of stage st and V of stage
  // st - 1 are done with, and the stages AHEAD of it go where they were.  A wave
  // alone refills a slot as soon as it has read it.  Loads are issued in the
  // order K 0, V 0, K 1, V 1, K 2, ...
  if (ns > 0) {
    constexpr auto most = [](int n) constexpr { return n < 63 ? n : 63; };
    auto held = [&](int slot) {   // page ids that came with the K stage in `slot`
      return [&, slot](int i) { return *(const int*)(ring + slot + G::PART + G::SCB + 4 * q_row(i)); };
    };
    // the first stages' ids before any of their loads: a wait for an id is one
    // for every load before it
    int first_ids[G::NST][G::QI + G::SI];
#pragma unroll
    for (int st = 0; st < G::NST; ++st)
#pragma unroll
      for (int i = 0; i < G::QI + G::SI; ++i) first_ids[st][i] = *entry(st < ns ? st : 0, q_row(i));
    if constexpr (G::F16) q_to_f16(q);
#pragma unroll
    for (int st = 0; st < G::NST; ++st)
      if (st < ns) {
        if (st > 0) issue_v(v_slot(st - 1));
        issue_k(st, k_slot(st), [&](int i) { return first_ids[st][i]; });
      }
    if (ns < G::NST) issue_v(v_slot(0));
    if (G::NST <= ns) wait_vm<most((G::NST - 1) * G::PW)>();
    else wait_vm<0>();
    if constexpr (G::WR > 1) lds_barrier();
    else asm volatile("" ::: "memory");
    scores s0, s1;
    products(std::integral_constant<int, k_slot(0)>{}, s0);
    finish(0, std::integral_constant<int, k_slot(0)>{}, s0);
    if constexpr (G::WR == 1) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (G::NST <= ns) issue_v(v_slot(1));
      if (G::NST < ns) issue_k(G::NST, k_slot(0), held(k_slot(0)));
    }
    // stage st, whose slots are i = st % 2; the next one's are 1 - i
    auto iterate = [&](int st, auto parity, scores& sa, scores& sb) {
      constexpr int i = decltype(parity)::value, j = 1 - i;
      // the later stages' loads may be outstanding
      if (st + G::AHEAD < ns) wait_vm<most((G::AHEAD - 1) * G::PW)>();
      else wait_vm<0>();
      auto refill = [&](int k_to, int v_to) {
        if (st + G::AHEAD < ns) issue_v(v_to);
        if (st + 1 + G::AHEAD < ns) issue_k(st + 1 + G::AHEAD, k_to, held(k_slot(j)));
      };
      if constexpr (G::WR > 1) {
        lds_barrier();
        refill(k_slot(i), v_slot(j));
      } else {
        asm volatile("" ::: "memory");
      }
      step(std::integral_constant<int, k_slot(j)>{}, std::integral_constant<int, v_slot(i)>{}, sa, sb);
      if (st + 1 < ns) finish(st + 1, std::integral_constant<int, k_slot(j)>{}, sb);
      if constexpr (G::WR == 1) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        refill(k_slot(j), v_slot(i));
      }
    };
    for (int st = 0; st < ns; st += 2) {
      iterate(st, std::integral_constant<int, 0>{}, s0, s1);
      if (st + 1 < ns) iterate(st + 1, std::integral_constant<int, 1>{}, s1, s0);
    }
  }

  // ---- join the lane groups' sums and the key groups' parts, and write
  const float v_unit = G::F16 ? a.c.v_unit : 1.0f, up2 = G::F16 ? kUp : 0.0f;
#pragma unroll
  for (int x = G::MT; x < 64; x <<= 1) l += __shfl_xor(l, x);
  if constexpr (G::WK == 1) {
    if (!live) return;
    const float inv = (l > 0.0f ? 1.0f / l : l) * v_unit;   // l: 0, or NaN kept
    const float lse2 = l == 0.0f ? -__builtin_inff() : m - up2 + __builtin_amdgcn_logf(l);
    const size_t ps = pc.part + at;
#pragma unroll
    for (int d = 0; d < G::DT; ++d)
#pragma unroll
      for (int i4 = 0; i4 < AN / 4; ++i4) {
        const int d4 = d * G::MT + 8 * i4 + 4 * g;
        const v4f y = {o[d][4 * i4] * inv, o[d][4 * i4 + 1] * inv, o[d][4 * i4 + 2] * inv, o[d][4 * i4 + 3] * inv};
        if (pc.direct)
          *(v2i*)(a.out + at * G::D + d4) = v2i{(int)pack_bf16(y[0], y[1]), (int)pack_bf16(y[2], y[3])};
        else if (ns > 0)
          *(v4f*)(a.part_o + ps * G::D + d4) = y;
      }
    if (g == 0 && pc.direct && a.lse) a.lse[at] = lse2 * kLn2;
    if (g == 0 && !pc.direct) a.part_lse[ps] = lse2;
  } else {
    float* const so = (float*)lds;                          // [WK][ROWS][SO]
    float* const sm = so + G::WK * G::ROWS * G::SO;         // [2][WK][ROWS]: m, l
    __syncthreads();                                        // the ring is no longer read
    if (g == 0) {
      sm[wk * G::ROWS + rl] = m;
      sm[(G::WK + wk) * G::ROWS + rl] = l;
    }
#pragma unroll
    for (int d = 0; d < G::DT; ++d)
#pragma unroll
      for (int i4 = 0; i4 < AN / 4; ++i4)
        *(v4f*)(so + (wk * G::ROWS + rl) * G::SO + d * G::MT + 8 * i4 + 4 * g) =
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
        const v4f y = *(const v4f*)(so + (x * G::ROWS + rw) * G::SO + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) ov[i] += y[i] * f;
      }
      const float inv = (ll > 0.0f ? 1.0f / ll : ll) * v_unit;
      const float lse2 = ll == 0.0f ? -__builtin_inff() : mm - up2 + __builtin_amdgcn_logf(ll);
      const size_t ar = a.even && !pc.direct ? 0 : (size_t)(t0 + rg / a.group) * a.heads + kvh * a.group + rg % a.group;
      if (pc.direct) {
        *(v2i*)(a.out + ar * G::D + d) = v2i{(int)pack_bf16(ov[0] * inv, ov[1] * inv),
                                             (int)pack_bf16(ov[2] * inv, ov[3] * inv)};
        if (d == 0 && a.lse) a.lse[ar] = lse2 * kLn2;
      } else {
        const v4f y = {ov[0] * inv, ov[1] * inv, ov[2] * inv, ov[3] * inv};
        if (a.even) {
          put_part(a, pc.part + rw, d, G::D, y, lse2);
        } else {
          const size_t ps = pc.part + ar;
          if (ns > 0) *(v4f*)(a.part_o + ps * G::D + d) = y;
          if (d == 0) a.part_lse[ps] = lse2;
        }
      }
    }
    // the workgroup that ends a segment's last piece joins them all
    if (a.even && !pc.direct) {
      int* const last = (int*)(sm + 2 * G::WK * G::ROWS);
      uint32_t* const count = a.counters + pc.req * a.c.kv_heads + kvh;
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // this wave's part is written
      __syncthreads();
      if (threadIdx.x == 0) {
        const uint32_t before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *last = before + 1 == (uint32_t)pc.pieces;
        if (*last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);   // for the next call
      }
      __syncthreads();
      if (!*last) return;
      const size_t first = pc.part - (size_t)pc.index * G::ROWS;
      constexpr int N = G::ROWS * LPR / G::THREADS;         // a thread's rows, THREADS / LPR apart
      static_assert(G::THREADS % LPR == 0, "one d per thread");
      const int rw0 = threadIdx.x / LPR, d0 = (threadIdx.x % LPR) * 4;
      int d[N];
#pragma unroll
      for (int k = 0; k < N; ++k) d[k] = d0;
      float mm[N], ll[N];
      v4f ov[N];
      auto row_of = [&](int i, int k) {                     // a row that is not there reads the first
        const int rw = rw0 + k * (G::THREADS / LPR);
        return first + (size_t)i * G::ROWS + (rw < n * a.group ? rw : 0);
      };
      join_parts<true, N, (N < 16 ? 16 / N : 1)>(a, pc.pieces, d, G::D, row_of, mm, ll, ov);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int rw = rw0 + k * (G::THREADS / LPR);
        if (rw < n * a.group)
          put_joined(a, (size_t)(t0 + rw / a.group) * a.heads + kvh * a.group + rw % a.group, d0, G::D, ov[k], mm[k],
                     ll[k]);
      }
    }
  }
}

// The request whose context is the want-th longest (in batches of up to 64
// requests, one per lane; in larger ones the want-th).
__device__ __forceinline__ int ranked_request(const AttnArgs& a, int want) {
  if (a.b.requests > 64) return want;
  const int lane = threadIdx.x & 63;
  const int kv = lane < a.b.requests ? a.b.kv_lens[lane] : 0;
  int rank = 0;
  for (int r = 0; r < a.b.requests; ++r) {
    const int other = __builtin_amdgcn_readlane(kv, r);
    rank += other > kv || (other == kv && r < lane);
  }
  return __builtin_ctzll(__ballot(lane < a.b.requests && rank == want));
}

template <class G>
__global__ __launch_bounds__(G::THREADS, G::MINW) void k_attn(AttnArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  Piece pc;
  if constexpr (G::EVEN) {
    if (a.even) {
      const Found f = find_piece(a, G::TT, G::MIN_TILES, blockIdx.x);
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
      pc.pieces = f.pieces;
      pc.index = i;
      attend<G>(a, pc, lds);
      return;
    }
  }
  // One row tile, those with the most keys first, so that short ones end the
  // launch: requests from the longest context on, row tiles from the last to
  // the first.  The kv head runs fastest: workgroups that share keys are 8 apart
  // where the heads are a multiple of 8 and meet in one XCD's L2.
  const int tiles = (int)(gridDim.x / a.splits) / (a.b.requests * a.c.kv_heads);
  int x = blockIdx.x;
  pc.kvh = x % a.c.kv_heads;
  x /= a.c.kv_heads;
  const int split = x % a.splits;
  x /= a.splits;
  const int tile = tiles - 1 - x % tiles;
  pc.req = ranked_request(a, x / tiles);
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
  if constexpr (G::WIDE) pc.kv = pc.kv < a.wide_keys ? pc.kv : a.wide_keys;   // (rows keep their places)
  pc.tiles = key_tiles(pc.p_lo, last_key<G>(a, pc.p_hi), a.window, a.sinks, G::TT);
  const int per = (pc.tiles.total + a.splits - 1) / a.splits;
  pc.s0 = split * per < pc.tiles.total ? split * per : pc.tiles.total;
  pc.s1 = pc.s0 + per < pc.tiles.total ? pc.s0 + per : pc.tiles.total;
  pc.direct = a.splits == 1;
  pc.part = (size_t)split * a.b.tokens * a.heads;
  attend<G>(a, pc, lds);
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
  float mm[1], ll[1];
  v4f ov[1];
  join_parts<false, 1, 8>(a, a.splits, {d}, D, [&](int s, int) { return s * rows + at; }, mm, ll, ov);
  put_joined(a, at, d, D, ov[0], mm[0], ll[0]);
}

template <class G>
hipError_t run(const AttnArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const hipError_t e = allow_lds((const void*)k_attn<G>, G::LDS, allowed);
  if (e != hipSuccess) return e;
  const int pairs = a.b.requests * a.c.kv_heads;
  if (a.even) {
    hipLaunchKernelGGL((k_attn<G>), dim3(a.groups), dim3(G::THREADS), G::LDS, st, a);
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

// Widens the pages of an NVFP4 cache that some new token of a request can see to
// fp16, which holds code times scale exactly, and writes the table that names them: a
// workgroup per page and 1024 lanes' work, 8 values of a row per lane.  Bound by HBM's writes.
template <int D>
__global__ __launch_bounds__(256) void k_widen(AttnArgs a) {
  constexpr int LPR = D / 8;
  const int req = blockIdx.x / a.wide_pages, j = blockIdx.x % a.wide_pages;
  if (threadIdx.x == 0 && blockIdx.y == 0) a.wide_table[blockIdx.x] = blockIdx.x;
  const Span span = token_span(a.b.q_start, req, a.b.tokens);
  const int kv = kv_bound(a.b.kv_lens[req], a.b.max_pages, a.c.page_shift);
  const int page_size = 1 << a.c.page_shift, first = j << a.c.page_shift;
  if (span.n <= 0 || first >= kv) return;
  const KeyRange range = key_range(kv - span.n, kv - 1, a.window, a.sinks);
  if (first + page_size - 1 <= range.from && first >= range.sinks) return;
  const int id = a.b.table[req * a.b.table_stride + j];
  const bool there = page_there(id, a.c.num_pages);
  const int items = page_size * a.c.kv_heads * LPR;
  const int64_t out = (int64_t)blockIdx.x * items * 16;
  uint8_t* const v_pool = a.wide + (int64_t)a.b.requests * a.wide_pages * items * 16;
#pragma unroll 4
  for (int it = blockIdx.y * 256 + threadIdx.x; it < items; it += 256 * gridDim.y) {
    const int i = it % LPR, row = it / LPR, head = row >> a.c.page_shift, key = row & (page_size - 1);
    const uint64_t at = there ? row_offset(key, id, a.c.page_shift, a.c.page, a.c.token) + head * a.c.head + 4 * i : 0;
    const uint64_t s_at = there ? row_offset(key, id, a.c.page_shift, a.c.s_page, a.c.s_token) + head * a.c.s_head + i / 2 : 0;
    uint32_t code[2] = {0, 0}, sc[2] = {0, 0};
    if (there) {
      code[0] = *(const uint32_t*)(a.c.k + at);
      code[1] = *(const uint32_t*)(a.c.v + at);
      sc[0] = ((const uint8_t*)a.c.k_scale)[s_at];
      sc[1] = ((const uint8_t*)a.c.v_scale)[s_at];
    }
#pragma unroll
    for (int kv2 = 0; kv2 < 2; ++kv2) {
      v2h s0, s1;
      e4m3x2_scales(sc[kv2], s0, s1);
      *(v8h*)((kv2 ? v_pool : a.wide) + out + (int64_t)it * 16) = e2m1x8_to_f16(code[kv2], s0);
    }
  }
}

// The kernel for a call whose largest request has `rows` rows per kv head.
// Up to 16 and 32 rows each wave takes all of them and a part of the keys,
// without barriers; up to 64, two waves share the keys of two; beyond, four
// waves of 32 rows share every key tile.  Against the next kernel, us:
//   16-row tiles: one token of one request over 131072 keys 92 (98), E4M3, four
//     requests 153 (158), 16 x 13 rows of one query head a kv head 38.4 (39.2);
//   32 rows: 16 x 13 tokens x 2 heads over 4096 keys 44.9 (47.6);
//   64 rows: 16 x 13 x 4 over 4096 keys 49.7 (54.5), 64 x 13 x 4 over 8192 in
//     E4M3 195 (272); a 13-row window of 1024 at head size 64 19.6 (21.9).
// At most 160 KB of LDS: two key waves for bf16 rows of 256, which have no 32-row
// kernel either (its registers do not fit).  64-key stages where the registers
// and two workgroups a CU allow them (E4M3 at 128: 198 -> 189; bf16 would leave
// one workgroup a CU: 40 x 13 rows over 4096 keys 99 -> 131).  Three waves a SIMD
// at head size 64 for many rows (309 against 348), two for up to 64 (20.5, 22.8).
template <int D, int FMT, class F>
auto visit_rows(int64_t rows, F f) {
  constexpr bool KV8 = FMT == OCQ_CACHE_E4M3;
  if constexpr (FMT == kWidened) {
    return f(Geo<D, FMT, 32, 4, 1, D == 256 ? 32 : 64, D == 256 ? 1 : D == 64 ? 3 : 2>{});   // (kWideRows)
  } else if constexpr (FMT == OCQ_CACHE_NVFP4) {
    if (rows <= 16) return f(Geo<D, FMT, 16, 1, D == 256 ? 2 : 4, 64, D == 256 ? 1 : 2>{});
    if constexpr (D < 256)
      if (rows <= 32) return f(Geo<D, FMT, 32, 1, 4, D == 128 ? 32 : 64, 2>{});
    if (rows <= 64) return f(Geo<D, FMT, 32, 2, 2, 64, D == 256 ? 1 : 2>{});
    return f(Geo<D, FMT, 32, 4, 1, D == 256 ? 32 : 64, D == 256 ? 1 : 2>{});
  } else {
  if (rows <= 16) return f(Geo<D, FMT, 16, 1, D == 256 && !KV8 ? 2 : 4, 32, D == 256 ? 1 : 2>{});
  if constexpr (D < 256)
    if (rows <= 32) return f(Geo<D, FMT, 32, 1, 4, 32, 2>{});
  if (rows <= 64) return f(Geo<D, FMT, 32, 2, 2, KV8 && D == 128 ? 64 : 32, D == 256 ? 1 : 2>{});
  return f(Geo<D, FMT, 32, 4, 1, D == 256 ? 32 : 64, D == 256 ? 1 : D == 64 ? 3 : 2>{});
  }
}
template <int D, class F>
auto visit_format(int format, int64_t rows, F f) {
  return format == OCQ_CACHE_BF16 ? visit_rows<D, OCQ_CACHE_BF16>(rows, f)
         : format == OCQ_CACHE_E4M3 ? visit_rows<D, OCQ_CACHE_E4M3>(rows, f)
         : format == OCQ_CACHE_NVFP4 ? visit_rows<D, OCQ_CACHE_NVFP4>(rows, f) : visit_rows<D, kWidened>(rows, f);
}
template <class F>
auto visit(int dim, int format, int64_t rows, F f) {
  return dim == 64 ? visit_format<64>(format, rows, f) : dim == 128 ? visit_format<128>(format, rows, f)
                                                                    : visit_format<256>(format, rows, f);
}

}  // namespace

// How a call is laid out.
//  * All rows of a request in one tile and more keys than one piece: pieces,
//    for two workgroups' worth of LDS (or one) on every CU.  Against splits of
//    equal number, or none where there are 512 pairs: 16 x 13 x 4 rows over 4096
//    keys 49.7 us (60.3), 16 x 13 over 2048 38.8 (46.0), a window of 1024 19.6
//    (20.6); 512 equal pairs lose 1 to 2 %, a batch with one long context gains.
//  * Several row tiles per request but few in all: each tile's keys in equal
//    splits, none below four key tiles of the longest request.
//  * Else one workgroup per row tile, all its keys: enough of them to fill the
//    GPU by themselves, or at most four key tiles (a join takes longer than
//    those: 257 keys 8.7 us in all).
AttnPlan attn_plan(int tokens, int requests, int max_new, int max_kv, int heads, int kv_heads, int dim, int format,
                   int window, int sinks, int64_t cap) {
  const int64_t rows = (int64_t)max_new * (heads / kv_heads);
  int64_t keys = max_kv;
  if (window > 0 && (int64_t)window + sinks + max_new < keys) keys = (int64_t)window + sinks + max_new;
  return visit(dim, format, rows, [&](auto geo) {
    typedef decltype(geo) G;
    AttnPlan p{0, 1, 0, 0, 0};
    const int64_t pairs = (int64_t)requests * kv_heads, tiles = (rows + G::ROWS - 1) / G::ROWS;
    p.lanes = (double)pairs * (double)tiles * G::THREADS;
    const int64_t key_tiles = (keys + G::TT - 1) / G::TT;
    if (key_tiles <= G::MIN_TILES) return p;
    if (G::EVEN && requests <= kEvenRequests && pairs < 4 * G::RESIDENT && pairs <= OCQ_ATTENTION_COUNTERS &&
        pairs * (cap / G::TT + 1) < (1 << 30)) {
      p.even = 1;
      p.slots = G::RESIDENT;
      p.groups = (int)(2 * pairs > p.slots ? p.slots + pairs : p.slots);   // no fewer than there can be pieces
      p.part_rows = (size_t)p.groups * G::ROWS;
      p.lanes = (double)p.groups * G::THREADS;
      return p;
    }
    const int64_t groups = pairs * tiles, want = (kTargetGroups + groups - 1) / groups, most = key_tiles / kMinTiles;
    const int64_t s = want < most ? want : most;
    p.splits = (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
    p.part_rows = p.splits > 1 ? (size_t)p.splits * tokens * heads : 0;
    p.lanes *= p.splits;
    if (p.splits > 1 && (double)tokens * heads * (G::D / 4) + 256 > p.lanes)   // the join's
      p.lanes = (double)tokens * heads * (G::D / 4) + 256;
    return p;
  });
}

int launch_attn(const AttnArgs& codes, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  AttnArgs a = codes;
  if (a.wide) {
    const int64_t lanes = ((int64_t)a.c.kv_heads << a.c.page_shift) * a.dim / 8;
    const int64_t ways = lanes / 1024 < 1 ? 1 : lanes / 1024 > 64 ? 64 : lanes / 1024;
    const dim3 grid((unsigned)(a.b.requests * a.wide_pages), (unsigned)ways), block(256);
    if (a.dim == 64) hipLaunchKernelGGL((k_widen<64>), grid, block, 0, st, codes);
    else if (a.dim == 128) hipLaunchKernelGGL((k_widen<128>), grid, block, 0, st, codes);
    else hipLaunchKernelGGL((k_widen<256>), grid, block, 0, st, codes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    const int64_t row = a.dim * 2, head = row << a.c.page_shift, page = head * a.c.kv_heads;
    a.format = kWidened;
    a.c = CacheArgs{codes.wide, codes.wide + (int64_t)a.b.requests * a.wide_pages * page, nullptr, nullptr, head, 0,
                    (uint32_t)page, (uint32_t)row, 0, 0, a.b.requests * a.wide_pages, codes.c.page_shift, codes.c.kv_heads,
                    codes.c.k_unit, codes.c.v_unit};
    a.b.table = codes.wide_table;
    a.b.table_stride = a.wide_pages;
  }
  return (int)visit(a.dim, a.format, (int64_t)a.max_new * a.group,
                    [&](auto geo) { return run<decltype(geo)>(a, st); });
}

}  // namespace ocq
