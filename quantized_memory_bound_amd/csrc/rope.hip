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

template <int DIM>
void run(const RopeArgs& a, hipStream_t st) {
  const int left = a.b.tokens - a.first;
  const dim3 grid(left < kAtOnce ? left : kAtOnce), block(kRopeThreads);
  if (a.e4m3) hipLaunchKernelGGL((k_rope<DIM, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_rope<DIM, false>), grid, block, 0, st, a);
}

}  // namespace

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
