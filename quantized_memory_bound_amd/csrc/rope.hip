// Rotary positions of q and k, and the append of k and v to a paged cache.
//
// Token i of a request's n new tokens stands at place p = kv_len - n + i of
// its context; its cache slot is page table[r][p / page_size], row p %
// page_size, and its rotary position is p too unless the caller gives one.
// With angle a_j = position * inv_freq[j], the pair (x_j, x_{j + rot/2}) or
// (x_2j, x_2j+1) becomes multiplier * (x_a cos a - x_b sin a,
// x_b cos a + x_a sin a); elements past rot are copied.
//
// The angle is reduced to a fraction of a turn in 64 bits (at position 10^6 a
// product in 32 bits would be off by a tenth of a radian), the sine and
// cosine are taken of that fraction in 32.  An E4M3 cache takes codes of the
// rotated 32-bit values with one scale per token and head, max / 448; a head with
// a value that is not finite has scale NaN, so that it stays visible.
//
// One workgroup per token: the token's rot/2 sines and cosines are made once,
// in LDS, for all heads.  A lane owns 16 elements of a head, both halves of
// its 8 pairs, so q_out may be q itself.  Bound by HBM: 4672 tokens of 48 heads of
// 128 elements 25.0 us (115 MB at 4.6 TB/s, a device copy's rate); 208 tokens into
// an E4M3 cache 5.6 us and one token 2.7 us by latency.
#include "layer_dev.h"
#include "layer_index.h"

namespace ocq {
namespace {

__device__ __forceinline__ void load8(const uint16_t* p, float* f) { unpack8_bf16(*(const v4i*)p, f); }
__device__ __forceinline__ void store8(uint16_t* p, const float* f) { *(v4i*)p = pack8_bf16(f); }

// The request of token t, or -1: the last r with q_start[r] <= t, found 64
// entries at a time (q_start does not fall).
__device__ __forceinline__ int request_of(const BatchArgs& b, int t) {
  const int lane = threadIdx.x & 63;
  int r = -1;
  for (int base = 0; base < b.requests; base += 64) {
    const int i = base + lane;
    const uint64_t m = __ballot(i < b.requests && b.q_start[i] <= t);
    r += __popcll(m);
    if (m != ~0ull) break;
  }
  if (r >= 0 && t >= b.q_start[r + 1]) r = -1;
  return r;
}

// The 16 values of a block of an NVFP4 row: its scale's code, then the codes.  The
// scale's E4M3 rounding decides first; the quotients are of the rounded scale.
struct Block4 {
  uint32_t scale;
  v2u codes;
};
__device__ __forceinline__ Block4 nvfp4_block(const float (&y)[16], float unit) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) amax = max_mag(amax, y[j]);
  Block4 b{0x7Fu, v2u{0u, 0u}};                    // E4M3's NaN
  if (!(amax < __builtin_inff())) return b;
  b.scale = enc_e4m3(amax / 6.0f / unit);
  if (b.scale == 0) return b;
  const float s = (float)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b.scale, 1.0f, false)[0] * unit;
  // Quotients by the reciprocal are within 2.5 units in the last place of fl32(y / s):
  // the same code unless a border lies that close.  From 1 on a border has 0x200000
  // in the 22 bits below the mantissa's first, below 1 it is an odd multiple of 1/4.
  // If any is that close, all are divided (one branch, rarely taken).
  const float rcp = 1.0f / s;   // (s a power of two times 8 to 15, far from overflow)
  float q[16];
  bool near = false;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    q[j] = y[j] * rcp;
    const float t = fabsf(q[j]) * 2.0f;
    near |= (t < 2.0f) & (fabsf(__builtin_amdgcn_fractf(t) - 0.5f) < 0x1p-20f);
    near |= (__float_as_uint(q[j]) & 0x3FFFFFu) - 0x1FFFFDu <= 6u;
  }
  if (near) {
    asm volatile("");
#pragma unroll
    for (int j = 0; j < 16; ++j) q[j] = y[j] / s;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t c = 0;
#pragma unroll
    for (int j = 8 * h; j < 8 * h + 8; ++j) q[j] = __builtin_amdgcn_fmed3f(q[j], -6.0f, 6.0f);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[8 * h], q[8 * h + 1], 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[8 * h + 2], q[8 * h + 3], 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[8 * h + 4], q[8 * h + 5], 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[8 * h + 6], q[8 * h + 7], 1.0f, 3);
    b.codes[h] = c;
  }
  return b;
}

// Sine and cosine of a (any finite size the positions give) in 64 bits: the turns a /
// 2 pi with 1 / 2 pi in two parts, so that the angle's own rounding is all that is
// lost, less the nearest quarter; the series of both within an eighth of a turn up
// to y^17 and y^16 (the next terms are below 2^-53); the quarter's signs and order.
__device__ __forceinline__ void sincos64(double a, double& sn, double& cs) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;   // 1 / 2 pi
  const double t = a * kHi, e = __builtin_fma(a, kHi, -t) + a * kLo;
  const double n = __builtin_rint(4.0 * (t - __builtin_rint(t)));
  const double y = ((t - __builtin_rint(t)) - 0.25 * n + e) * 6.283185307179586476925, z = y * y;
  double s = 1.0 / 355687428096000.0, c = 1.0 / 20922789888000.0;
  s = __builtin_fma(s, z, -1.0 / 1307674368000.0);
  s = __builtin_fma(s, z, 1.0 / 6227020800.0);
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  s = __builtin_fma(s * z, y, y);
  c = __builtin_fma(c, z, -1.0 / 87178291200.0);
  c = __builtin_fma(c, z, 1.0 / 479001600.0);
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  c = __builtin_fma(c, z, -0.5);
  c = __builtin_fma(c, z, 1.0);
  const int q = (int)n & 3;
  const double u = q & 1 ? c : s, v = q & 1 ? s : c;
  sn = q & 2 ? -u : u;
  cs = (q + 1) & 2 ? -v : v;
}

constexpr int kRopeThreads = 256, kAtOnce = kLanesAtOnce / kRopeThreads;   // tokens of a launch

template <int DIM, bool E4M3>
__global__ __launch_bounds__(kRopeThreads) void k_rope(RopeArgs a) {
  constexpr int LPH = DIM / 16;   // lanes per head
  __shared__ float s_cos[DIM / 2], s_sin[DIM / 2];
  const int t = a.first + blockIdx.x;
  const int r = request_of(a.b, t);
  if (r < 0) return;
  const int64_t place = (int64_t)a.b.kv_lens[r] - a.b.q_start[r + 1] + t;
  const int64_t pos = a.positions ? a.positions[t] : place;
  const int half = a.rot / 2;
  for (int j = threadIdx.x; j < half; j += kRopeThreads) {
    double turns = (double)pos * a.inv_freq[j] * 0.15915494309189533577;   // 1 / (2 pi)
    turns -= __builtin_rint(turns);
    float sn, cs;
    sincospif(2.0f * (float)turns, &sn, &cs);
    s_cos[j] = cs * a.multiplier;
    s_sin[j] = sn * a.multiplier;
  }
  lds_barrier();
  // the token's cache row; none if its place or page is not in the pool
  int page = -1;
  if (place >= 0 && place >> a.c.page_shift < a.b.max_pages)
    page = a.b.table[r * a.b.table_stride + (place >> a.c.page_shift)];
  const bool slot = page >= 0 && page < a.c.num_pages;
  const int key = slot ? (int)place : 0;
  page = slot ? page : 0;
  const int kvh = a.c.kv_heads, items = (a.heads + 2 * kvh) * LPH;
  for (int it = threadIdx.x; it < items; it += kRopeThreads) {
    int head = it / LPH;
    const int i = it % LPH;
    const int which = head < a.heads ? 0 : head < a.heads + kvh ? 1 : 2;   // q, k, v
    head -= which == 0 ? 0 : which == 1 ? a.heads : a.heads + kvh;
    const uint16_t* src = which == 0 ? a.q + t * a.q_token + head * a.q_head
                        : which == 1 ? a.k + t * a.k_token + head * a.k_head
                                     : a.v + t * a.v_token + head * a.v_head;
    const bool turn = i * 16 < a.rot;
    const bool split = turn && !a.interleaved;
    const int d0 = split ? 8 * i : 16 * i, d1 = split ? half + 8 * i : 16 * i + 8;
    float x[16];
    load8(src + d0, x);
    load8(src + d1, x + 8);
    if (which < 2 && turn) {
      const float* cs = s_cos + 8 * i;
      const float* sn = s_sin + 8 * i;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = cs[j], s = sn[j];
        if (a.interleaved) {
          const float u = x[2 * j], v = x[2 * j + 1];
          x[2 * j] = u * c - v * s;
          x[2 * j + 1] = v * c + u * s;
        } else {
          const float u = x[j], v = x[8 + j];
          x[j] = u * c - v * s;
          x[8 + j] = v * c + u * s;
        }
      }
    }
    if (which == 0) {
      uint16_t* dst = a.q_out + ((size_t)t * a.heads + head) * DIM;
      store8(dst + d0, x);
      store8(dst + d1, x + 8);
      continue;
    }
    uint8_t* pool = (which == 1 ? a.c.k : a.c.v) + row_offset(key, page, a.c.page_shift, a.c.page, a.c.token) +
                    head * a.c.head;
    if constexpr (!E4M3) {
      if (slot) {
        store8((uint16_t*)pool + d0, x);
        store8((uint16_t*)pool + d1, x + 8);
      }
    } else {
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = max_mag(amax, x[j]);
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) amax = max_mag(amax, __shfl_xor(amax, o));
      const float s = e4m3_scale(amax);
      float y[2][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[0][j] = x[j];
        y[1][j] = x[8 + j];
      }
      const Quot qt = e4m3_quot_of(s, y);
      const v2u c0 = s > 0.0f ? e4m3x8_quot(y[0], qt.s, qt.rcp) : v2u{0u, 0u};
      const v2u c1 = s > 0.0f ? e4m3x8_quot(y[1], qt.s, qt.rcp) : v2u{0u, 0u};
      if (slot) {
        *(v2u*)(pool + d0) = c0;
        *(v2u*)(pool + d1) = c1;
        if (i == 0)
          (which == 1 ? a.c.k_scale : a.c.v_scale)[row_offset(key, page, a.c.page_shift, a.c.s_page, a.c.s_token) +
                                                   head * a.c.s_head] = s;
      }
    }
  }
}

// The same into an NVFP4 cache, `per` tokens a workgroup: each wave finds one
// token's slot and makes its sines and cosines, in 64 bits; then all lanes take the
// tokens' heads.  An item of q is as above; one of k or v is a block of 16 elements,
// which reads what it needs of its pairs' other halves (eight elements in a row
// are all first or all second ones).  Four tokens a workgroup where there are many:
// 4672 tokens of 48 heads of 128 elements 26.2 us instead of 31.2 (a copy of the same
// bytes: 21), 208 tokens 11.4 instead of 6.4.
constexpr int kAppendTokens = 4, kAppendMany = 1024;   // from so many tokens on

struct Slot {
  int t, page, key;          // token (-1: none), its page (-1: not appended) and place
};

template <int DIM>
__global__ __launch_bounds__(kRopeThreads) void k_rope4(RopeArgs a, int per) {
  constexpr int LPH = DIM / 16;   // items of a head
  __shared__ double s_cos[kAppendTokens][DIM / 2], s_sin[kAppendTokens][DIM / 2];
  __shared__ Slot s_slot[kAppendTokens];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = a.rot / 2;
  const int t0 = a.first + blockIdx.x * per;
  if (wave < per) {
    const int t = t0 + wave, r = t < a.b.tokens ? request_of(a.b, t) : -1;
    Slot sl{-1, -1, 0};
    if (r >= 0) {
      const int64_t place = (int64_t)a.b.kv_lens[r] - a.b.q_start[r + 1] + t;
      const int64_t pos = a.positions ? a.positions[t] : place;
      sl.t = t;
      if (place >= 0 && place >> a.c.page_shift < a.b.max_pages) {
        const int page = a.b.table[r * a.b.table_stride + (place >> a.c.page_shift)];
        if (page_there(page, a.c.num_pages)) {
          sl.page = page;
          sl.key = (int)place;
        }
      }
      for (int j = lane; j < half; j += 64) {
        double sn, cs;
        sincos64((double)pos * a.inv_freq[j], sn, cs);
        s_cos[wave][j] = cs * a.multiplier;
        s_sin[wave][j] = sn * a.multiplier;
      }
    }
    if (lane == 0) s_slot[wave] = sl;
  }
  lds_barrier();
  const int kvh = a.c.kv_heads, items = (a.heads + 2 * kvh) * LPH;
  for (int x = threadIdx.x; x < per * items; x += kRopeThreads) {
    const int w = x / items, it = x - w * items;
    const Slot sl = s_slot[w];
    if (sl.t < 0) continue;
    const int t = sl.t, i = it % LPH;
    int head = it / LPH;
    const int which = head < a.heads ? 0 : head < a.heads + kvh ? 1 : 2;   // q, k, v
    head -= which == 0 ? 0 : which == 1 ? a.heads : a.heads + kvh;
    const uint16_t* const src = which == 0 ? a.q + t * a.q_token + head * a.q_head
                              : which == 1 ? a.k + t * a.k_token + head * a.k_head
                                           : a.v + t * a.v_token + head * a.v_head;
    const double* const dc = s_cos[w];
    const double* const ds = s_sin[w];
    const bool turn = i * 16 < a.rot;
    if (which == 0) {
      const bool split = turn && !a.interleaved;
      const int d0 = split ? 8 * i : 16 * i, d1 = split ? half + 8 * i : 16 * i + 8;
      float y[16];
      load8(src + d0, y);
      load8(src + d1, y + 8);
      if (turn) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float c = (float)dc[8 * i + j], s = (float)ds[8 * i + j];
          if (a.interleaved) {
            const float u = y[2 * j], v = y[2 * j + 1];
            y[2 * j] = u * c - v * s;
            y[2 * j + 1] = v * c + u * s;
          } else {
            const float u = y[j], v = y[8 + j];
            y[j] = u * c - v * s;
            y[8 + j] = v * c + u * s;
          }
        }
      }
      uint16_t* const dst = a.q_out + ((size_t)t * a.heads + head) * DIM;
      store8(dst + d0, y);
      store8(dst + d1, y + 8);
      continue;
    }
    if (sl.page < 0) continue;
    float y[16];
    load8(src + 16 * i, y);
    load8(src + 16 * i + 8, y + 8);
    if (which == 1 && turn) {
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double c = dc[8 * i + j], s = ds[8 * i + j], u = y[2 * j], v = y[2 * j + 1];
          y[2 * j] = (float)(u * c - v * s);
          y[2 * j + 1] = (float)(v * c + u * s);
          if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // not all 64-bit values at once
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = 16 * i + 8 * h;
          const bool first = e < half;
          float o[8];
          load8(src + (first ? e + half : e - half), o);
          const double* const cs = dc + (first ? e : e - half);
          const double* const sn = ds + (first ? e : e - half);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const double u = (double)y[8 * h + j] * cs[j], v = (double)o[j] * sn[j];
            y[8 * h + j] = (float)(first ? u - v : u + v);
            if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // not all 64-bit values at once
          }
        }
      }
    }
    const Block4 b = nvfp4_block(y, which == 1 ? a.c.k_unit : a.c.v_unit);
    uint8_t* const pool = (which == 1 ? a.c.k : a.c.v) + head * a.c.head +
                          row_offset(sl.key, sl.page, a.c.page_shift, a.c.page, a.c.token);
    uint8_t* const sc = (uint8_t*)(which == 1 ? a.c.k_scale : a.c.v_scale) + head * a.c.s_head +
                        row_offset(sl.key, sl.page, a.c.page_shift, a.c.s_page, a.c.s_token);
    *(v2u*)(pool + 8 * i) = b.codes;
    sc[i] = (uint8_t)b.scale;
  }
}

template <int DIM>
void run(const RopeArgs& a, hipStream_t st) {
  const int left = a.b.tokens - a.first, now = left < kAtOnce ? left : kAtOnce;
  const dim3 block(kRopeThreads);
  if (a.format == OCQ_CACHE_NVFP4) {
    const int per = a.b.tokens >= kAppendMany ? kAppendTokens : 1;
    hipLaunchKernelGGL((k_rope4<DIM>), dim3((now + per - 1) / per), block, 0, st, a, per);
  } else if (a.format == OCQ_CACHE_E4M3) {
    hipLaunchKernelGGL((k_rope<DIM, true>), dim3(now), block, 0, st, a);
  } else {
    hipLaunchKernelGGL((k_rope<DIM, false>), dim3(now), block, 0, st, a);
  }
}

// The values of a pool of codes: a lane makes 8 of one row, of k, then of v, so that
// a wave's stores lie side by side (32,000 tokens of 8 heads of 128: 36.8 us; 16 a lane
// 44.9, with non-temporal stores 61).  Bound by HBM's writes.
template <bool NVFP4>
__global__ __launch_bounds__(256) void k_values(ValuesArgs a, int64_t first) {
  const int lanes = a.dim / 8;
  const int64_t it = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = it / lanes;
  if (row >= a.rows) return;
  const int i = (int)(it % lanes), key = (int)(row & ((1 << a.c.page_shift) - 1));
  const int64_t up = row >> a.c.page_shift;
  const int head = (int)(up % a.c.kv_heads), page = (int)(up / a.c.kv_heads);
  const uint64_t at = row_offset(key, page, a.c.page_shift, a.c.page, a.c.token) + head * a.c.head;
  const uint64_t s_at = row_offset(key, page, a.c.page_shift, a.c.s_page, a.c.s_token) + head * a.c.s_head;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint8_t* const pool = (kv ? a.c.v : a.c.k) + at;
    float y[8];
    if constexpr (NVFP4) {
      const uint32_t sc = ((const uint8_t*)(kv ? a.c.v_scale : a.c.k_scale))[s_at + i / 2];
      const float unit = kv ? a.c.v_unit : a.c.k_unit;
      v2h s0, s1;
      e4m3x2_scales(sc, s0, s1);
      const v8h v = e2m1x8_to_f16(*(const uint32_t*)(pool + 4 * i), s0);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = (float)v[j] * unit;
    } else {
      const v2u c = *(const v2u*)(pool + 8 * i);
      const float s = (kv ? a.c.v_scale : a.c.k_scale)[s_at];
      const v8h v = e4m3x8_to_f16(c[0], c[1]);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = (float)v[j] * s;
    }
    store8((kv ? a.v : a.k) + row * a.dim + 8 * i, y);
  }
}

}  // namespace

int launch_values(const ValuesArgs& a, void* stream) {
  const int64_t items = a.rows * (a.dim / 8);
  for (int64_t first = 0; first < items; first += kLanesAtOnce) {
    const int64_t left = items - first, now = left < kLanesAtOnce ? left : kLanesAtOnce;
    const dim3 grid((unsigned)((now + 255) / 256)), block(256);
    if (a.format == OCQ_CACHE_NVFP4) hipLaunchKernelGGL((k_values<true>), grid, block, 0, (hipStream_t)stream, a, first);
    else hipLaunchKernelGGL((k_values<false>), grid, block, 0, (hipStream_t)stream, a, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
  }
  return 0;
}

int launch_rope(const RopeArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  RopeArgs part = a;
  for (int64_t first = 0; first < a.b.tokens; first += kAtOnce) {
    part.first = (int)first;
    if (a.dim == 64) run<64>(part, st);
    else if (a.dim == 128) run<128>(part, st);
    else run<256>(part, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
  }
  return 0;
}

}  // namespace ocq
