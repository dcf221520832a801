// Which drafted tokens of a verify pass stay, and the token that follows them.
//
// Request r has rows t0 .. t0 + n - 1; row t gives the target's distribution p
// of the token after ids[t], and draft i of the request is ids[t0 + i + 1], drawn
// from the draft model's q (a row of `draft`; without one q is 1 at the draft).
// With l the row's logits, p_j = e_j / Z, e_j = exp((l_j - max l) / T), Z = sum_j
// e_j; T = 0: 1 at the first of the largest.  Draft i stays while u_i q(x) < p(x);
// at the first that does not, the next token is drawn from w = max(p - q, 0)
// (without q: from p without x), after the last one from w = p of its row: the
// lowest j with sum_{i <= j} w_i > u sum w.
//
// Two launches.  A reads all logits once: each row's maximum and sum Z', of 32-bit
// exponentials added eight at a time, then in 64 bits; the workgroup that ends a
// request's last row compares its drafts (64-bit exponentials with Z', off by less
// than 2^-19, see k_stats) and leaves what drawing needs.  B sums the
// drawn row's weights in 64 bits, in chunks; the workgroup that ends a request's
// last chunk finds the chunk and the place in it.  (With given probabilities there
// is no A: B's workgroups compare the drafts themselves.)
//
// The place that a random number falls on hangs on every weight before it, so Z' is
// not enough for w = max(e_j / Z - q_j, 0), and Z is known only when all chunks are.
// With S the j where e_j / Z' > q_j a chunk leaves sum e, sum_S e and sum_S q: its
// weights are sum_S e / Z - sum_S q but for those j that lie between Z' and Z, each of
// which is off by at most d e_j / Z, d = |Z' / Z - 1|.  It leaves the sum of e_j / Z'
// over all j within 2^-16 of the border as well; where d is larger or d times that
// sum is over 10^-10 of the weights (q is p but for roundings) the chunks are summed
// again with Z, by one workgroup.  Against a launch for Z before the weights': 3.9
// us.  What one workgroup leaves for another of its launch goes through
// device-scope stores and loads, past the L2s.
#include "kcommon.h"
#include "layer_index.h"
#include "step.h"

namespace ocq {

// A part of a row: its maximum and where it first stands; the sum of exp((l - max) /
// T), NaN where not every logit is a number.
struct RowStat {
  uint64_t top_at;   // float, int
  double sum;
};

// The draft after a row: its logit and id (-1: none), u q of it.
struct RowDraft {
  uint64_t logit_id;
  double uq;
};

// What a request draws its next token from.
struct Choice {
  double top, inv_t, z;      // of the drawn row (logits), z as A has it
  int64_t q_row;             // the draft's row that is subtracted, -1: none
  int t0, n, count;          // first row, rows, accepted drafts
  int draw;                  // 0: the next token is `next` (-1: none)
  int next;
  int without;               // the id that is left out, -1: none
};

namespace {

constexpr int kThreads = 256, kVec = 8;            // elements that a lane loads at once
constexpr double kLog2e = 1.4426950408889634074;

// eight elements from p, at any alignment (vector loads need none here)
__device__ __forceinline__ void load8(const float* p, float* f) {
  float v[8];
  __builtin_memcpy(v, p, 32);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = v[j];
}
__device__ __forceinline__ void load8(const uint16_t* p, float* f) {
  uint32_t v[4];
  __builtin_memcpy(v, p, 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(v[j] << 16);
    f[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// elements j .. j + 7 of a row, `none` past its end
template <class T>
__device__ __forceinline__ void load_row(const T* row, int j, int end, float none, float* f) {
  if (j + kVec <= end) {
    load8(row + j, f);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = j + i < end ? load1(row + j + i) : none;
  }
}

// elements of a row's part where `ways` workgroups share it
__device__ __forceinline__ int part_size(int vocab, int ways) { return ((vocab + ways - 1) / ways + kVec - 1) / kVec * kVec; }

// The request of token t, or -1 (64 of them at a time).
__device__ __forceinline__ int request_of(const DraftArgs& a, int t) {
  const int lane = threadIdx.x & 63;
  int r = -1;
  for (int base = 0; base < a.requests; base += 64) {
    const int i = base + lane;
    const uint64_t m = __ballot(i < a.requests && a.q_start[i] <= t);
    r += __popcll(m);
    if (m != ~0ull) break;
  }
  if (r >= 0 && t >= a.q_start[r + 1]) r = -1;
  return r;
}

__device__ __forceinline__ float temperature(const DraftArgs& a, int r) { return a.temps ? a.temps[r] : a.temp; }

// better of two (value, place): the larger, then the lower place
__device__ __forceinline__ void best(float& v, int& at, float v2, int at2) {
  const bool take = v2 > v || (v2 == v && at2 < at);
  v = take ? v2 : v;
  at = take ? at2 : at;
}

template <class V>
__device__ __forceinline__ V load_agent(const V* p) {
  return __builtin_bit_cast(V, __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}
template <class V>
__device__ __forceinline__ void store_agent(V* p, V v) {
  __hip_atomic_store((uint64_t*)p, __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// A request's counter: 128 requests' lie 128 bytes apart.  (Arrivals at one cache
// line follow each other 20 ns apart: side by side, 2080 of them took 30 us.)
__device__ __forceinline__ uint32_t* counter_of(const DraftArgs& a, int r) {
  static_assert(OCQ_ATTENTION_COUNTERS == 128 * 32, "");
  return a.counters + (r & 127) * 32 + (r >> 7);
}
// Whether this workgroup is the last of `all` to come here with this counter, for
// all its threads; what the others' first wave stored before is then visible to
// device-scope loads.  The counter is 0 again afterwards.
__device__ __forceinline__ bool last_of(uint32_t* counter, uint32_t all, int* shared) {
  if (threadIdx.x == 0) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint32_t before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *shared = before + 1 == all;
    if (*shared) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *shared != 0;
}

// A double of another lane (0 where there is none): DPP, no LDS round trip.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane64(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane) << 32 |
                                        (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane));
}
// Sums over the lanes before and with this one: within rows of 16 (row_shr 1, 2, 4,
// 8), then each row's last into the next rows (row_bcast 15 and 31).
__device__ __forceinline__ double scan64(double v) {
  v += dpp64<0x111, 0xF>(v);
  v += dpp64<0x112, 0xF>(v);
  v += dpp64<0x114, 0xF>(v);
  v += dpp64<0x118, 0xF>(v);
  v += dpp64<0x142, 0xA>(v);
  v += dpp64<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ double sum64(double v) { return lane64(scan64(v), 63); }

// e^y for y <= 0: 2^n times the series of e^g, g = (y log2 e - n) ln 2 within ln 2 /
// 2, up to g^11 / 11! (the next term is below 2^-47); 0 from 2^-1075 down, NaN kept.
__device__ __forceinline__ double exp64(double y) {
  double x = y * kLog2e;
  x = x < -1100.0 ? -1100.0 : x;
  const double n = __builtin_rint(x), g = (x - n) * 0.69314718055994530942;
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, g, 1.0 / 3628800.0);
  p = __builtin_fma(p, g, 1.0 / 362880.0);
  p = __builtin_fma(p, g, 1.0 / 40320.0);
  p = __builtin_fma(p, g, 1.0 / 5040.0);
  p = __builtin_fma(p, g, 1.0 / 720.0);
  p = __builtin_fma(p, g, 1.0 / 120.0);
  p = __builtin_fma(p, g, 1.0 / 24.0);
  p = __builtin_fma(p, g, 1.0 / 6.0);
  p = __builtin_fma(p, g, 0.5);
  p = __builtin_fma(p, g, 1.0);
  p = __builtin_fma(p, g, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// ---------------------------------------------------------------- which drafts stay

constexpr int kRows = kThreads / 16;    // rows of a request compared at a time
struct ChooseShared {
  double z[kRows];
  float top[kRows];
  int at[kRows], id[kRows], first;
};

// The draft's rows before request r's: one less than its tokens for each request
// (by whole waves).
__device__ __forceinline__ int64_t draft_rows_before(const DraftArgs& a, int r, int t0) {
  int idle = 0;
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < r; base += 64)
    idle += __popcll(__ballot(base + lane < r && token_span(a.q_start, base + lane, a.tokens).n <= 0));
  return t0 - (r - idle);
}

// The draft after row t = t0 + i of a request with n rows.
struct Draft {
  int x;
  float l;
  double uq;
};
template <class T, class Q>
__device__ __forceinline__ Draft draft_of(const DraftArgs& a, int t, int i, int n, int64_t before) {
  Draft d{-1, 0.0f, 0.0};
  if (i < n - 1) {
    const int x = a.ids[t + 1];
    if (x >= 0 && x < a.vocab) {
      const float q = !a.draft ? 1.0f : before + i >= 0 && before + i < a.draft_rows
                      ? load1((const Q*)a.draft + (before + i) * a.d_stride + x) : __builtin_nanf("");
      d = Draft{x, load1((const T*)a.target + t * a.t_stride + x), (double)a.u_accept[t] * (double)q};
    }
  }
  return d;
}

// By all threads of a workgroup; 16 lanes share a row's parts (64 at most).
template <class T, class Q, bool PROBS>
__device__ __forceinline__ Choice choose(const DraftArgs& a, int r, const Span& sp, int64_t before, float temp,
                                         ChooseShared& sh) {
  const int n = sp.n < 0 ? 0 : sp.n;
  const double inv_t = 1.0 / (double)temp;
  Choice c{0.0, inv_t, 0.0, -1, sp.t0, n, 0, 1, -1, -1};
  for (int i0 = 0; i0 < n; i0 += kRows) {
    const int row = threadIdx.x >> 4, i = i0 + row, t = sp.t0 + (i < n ? i : 0);
    Draft d;
    if constexpr (PROBS) {
      d = draft_of<T, Q>(a, t, i, n, before);
    } else {
      const uint64_t li = load_agent(&a.row_drafts[t].logit_id);
      d = Draft{i < n ? (int)(li >> 32) : -1, __uint_as_float((uint32_t)li), load_agent(&a.row_drafts[t].uq)};
    }
    float top = -__builtin_inff();
    int at = 0x7FFFFFFF;
    double z = 0.0;
    if constexpr (!PROBS) {
      const RowStat* const st = a.stats + (size_t)t * a.splits;
      uint64_t ta[4];
      double part[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {      // all of them on their way together
        const int k = (threadIdx.x & 15) + 16 * b;
        ta[b] = load_agent(&st[k < a.splits ? k : 0].top_at);
        part[b] = load_agent(&st[k < a.splits ? k : 0].sum);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) best(top, at, __uint_as_float((uint32_t)ta[b]), (int)(ta[b] >> 32));
#pragma unroll
      for (int b = 1; b < 16; b <<= 1) best(top, at, __shfl_xor(top, b), __shfl_xor(at, b));
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float v = __uint_as_float((uint32_t)ta[b]);
        if ((int)(threadIdx.x & 15) + 16 * b < a.splits)
          z += temp == 0.0f || part[b] == 0.0 ? part[b] : part[b] * exp64(((double)v - (double)top) * inv_t);
      }
#pragma unroll
      for (int b = 1; b < 16; b <<= 1) z += __shfl_xor(z, b);
    }
    bool keep = false;
    if (d.x >= 0) {
      if (PROBS) keep = d.uq < (double)d.l;
      else if (temp == 0.0f) keep = z == 0.0 && d.uq < (d.x == at ? 1.0 : 0.0);
      else keep = d.uq * z < exp64(((double)d.l - (double)top) * inv_t);
    }
    if (threadIdx.x == 0) sh.first = 0x7FFFFFFF;
    __syncthreads();
    if (i < n && !keep && (threadIdx.x & 15) == 0) atomicMin(&sh.first, i);
    if ((threadIdx.x & 15) == 0) {
      sh.z[row] = z;
      sh.top[row] = top;
      sh.at[row] = at;
      sh.id[row] = d.x;
    }
    __syncthreads();
    const int first = sh.first;
    if (first != 0x7FFFFFFF) {       // (the row after the last draft keeps none)
      c.count = first;
      c.top = (double)sh.top[first - i0];
      c.z = sh.z[first - i0];
      if (first < n - 1) {
        if (a.draft) c.q_row = before + first >= 0 && before + first < a.draft_rows ? before + first : -1;
        else c.without = sh.id[first - i0];
      }
      if (!PROBS && temp == 0.0f) {
        c.draw = 0;
        c.next = sh.z[first - i0] == 0.0 && sh.at[first - i0] != 0x7FFFFFFF ? sh.at[first - i0] : -1;
      }
      break;
    }
    __syncthreads();
  }
  if (n == 0) c.draw = 0;
  return c;
}

// A request's rows: the accepted drafts, the next token if it is known, -1.
__device__ __forceinline__ void put_rows(const DraftArgs& a, const Choice& c, int r) {
  for (int i = threadIdx.x; i < c.n; i += kThreads)
    if (i != c.count || !c.draw) a.out[c.t0 + i] = i < c.count ? a.ids[c.t0 + i + 1] : i == c.count ? c.next : -1;
  if (threadIdx.x == 0) a.accepted[r] = c.count;
}

// ---------------------------------------------------------------- A: statistics of every row

// A lane's vector as it lies in memory, and the one that changes nothing.
template <class T>
struct Raw {
  static constexpr int W = kVec * sizeof(T) / 4;
  uint32_t w[W];
};
__device__ __forceinline__ void unpack(const Raw<float>& r, float* f) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void unpack(const Raw<uint16_t>& r, float* f) {
#pragma unroll
  for (int i = 0; i < kVec / 2; ++i) {
    f[2 * i] = __uint_as_float(r.w[i] << 16);
    f[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
}

// The statistics of one row's part.  UNR vectors of a lane are summed while the
// next UNR are on their way.
//
// How far Z' is off, in units of 2^-24 of it: an exponential 2^((l - top) c), with y =
// (top - l) / T, has y from the difference, y from c's rounding, y from the product's
// and 2 from the instruction; eight of them added in pairs 3.  The mean of y over a
// lane's n elements, by weight, is below the w with w e^w = n / e (one likely one
// beside n unlikely ones), 8.1 at the most that there can be, 2^16: 30 in all.  Sums
// across vectors, and what a new maximum multiplies them by, are 64-bit: in 32 a
// long tail of small terms is lost one by one (131072 logits of a row, 256 of 0 and
// all others -18.75: 2^-18 of Z').  208 rows of 131072 with the drawn rows 30.4 us a
// call, with sums in 32 bits 29.7.
template <class T, class Q>
__global__ __launch_bounds__(kThreads) void k_stats(DraftArgs a) {
  constexpr int UNR = sizeof(T) == 2 ? 4 : 2, STEP = kThreads * kVec, TILE = UNR * STEP;
  __shared__ ChooseShared sh;
  __shared__ float s_top[4];
  __shared__ int s_at[4], s_last;
  __shared__ double s_sum[4];
  const int t = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int per = part_size(a.vocab, a.splits);
  const int from = split * per, end = from + per < a.vocab ? from + per : a.vocab;
  const T* const row = (const T*)a.target + t * a.t_stride;
  Raw<T> raw[UNR];
  auto load = [&](int j) {       // whole vectors; those that the row's end cuts come last
#pragma unroll
    for (int k = 0; k < UNR; ++k) {
      if (j + k * STEP + kVec <= end) {
        __builtin_memcpy(raw[k].w, row + j + k * STEP, sizeof(raw[k].w));
      } else {
#pragma unroll
        for (int i = 0; i < Raw<T>::W; ++i) raw[k].w[i] = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;   // -inf
      }
    }
  };
  const int j0 = from + threadIdx.x * kVec;
  load(j0);
  if (blockIdx.x == 0)                                  // requests without rows
    for (int r = threadIdx.x; r < a.requests; r += kThreads)
      if (token_span(a.q_start, r, a.tokens).n <= 0) a.accepted[r] = 0;
  const int cut = end - end % kVec + threadIdx.x;
  const float rest = (int)threadIdx.x < end % kVec ? load1(row + cut) : -__builtin_inff();
  const int r = request_of(a, t);
  if (r < 0) {
    if (threadIdx.x == 0 && split == 0) a.out[t] = -1;
    return;
  }
  const float temp = temperature(a, r);
  const Span sp = token_span(a.q_start, r, a.tokens);
  // what the request's comparisons take of this row's draft, on its way early
  const int64_t before = a.draft ? draft_rows_before(a, r, sp.t0) : 0;
  Draft d{-1, 0.0f, 0.0};
  if (split == 0 && threadIdx.x == 0) d = draft_of<T, Q>(a, t, t - sp.t0, sp.n, before);
  float top = rest;
  int at = (int)threadIdx.x < end % kVec && rest > -__builtin_inff() ? cut : 0x7FFFFFFF;
  double sum = 0.0;
  if (temp == 0.0f) {
    bool bad = rest != rest;
    if (bad) top = -__builtin_inff();
    for (int j = j0; j < end; j += TILE) {
      Raw<T> now[UNR];
#pragma unroll
      for (int k = 0; k < UNR; ++k) now[k] = raw[k];
      if (j + TILE < end) load(j + TILE);
#pragma unroll
      for (int k = 0; k < UNR; ++k) {
        // the vector's maximum first: its place only where it is a new one
        float f[kVec], m;
        unpack(now[k], f);
        m = f[0];
        bool nan = f[0] != f[0];
#pragma unroll
        for (int i = 1; i < kVec; ++i) {
          m = fmaxf(m, f[i]);
          nan |= f[i] != f[i];
        }
        bad |= nan;
        if (m > top || (m == top && j + k * STEP < at)) {
          top = m;
#pragma unroll
          for (int i = kVec - 1; i >= 0; --i)
            if (f[i] == m) at = j + k * STEP + i;
        }
      }
    }
    if (top == -__builtin_inff()) at = 0x7FFFFFFF;
    if (bad) sum = __builtin_nan("");
  } else {
    const float c = fminf((float)(kLog2e / (double)temp), 1e30f);   // (finite at any T > 0: 0 times it is 0)
    const double inv_t = 1.0 / (double)temp;
    sum = rest == -__builtin_inff() ? 0.0 : 1.0 + 0.0 * (double)rest;   // e^0; NaN and inf are none
    if (rest != rest) top = -__builtin_inff();
    for (int j = j0; j < end; j += TILE) {
      float f[UNR][kVec], m = top;
#pragma unroll
      for (int k = 0; k < UNR; ++k) unpack(raw[k], f[k]);
      if (j + TILE < end) load(j + TILE);
#pragma unroll
      for (int k = 0; k < UNR; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) m = fmaxf(m, f[k][i]);
      if (m > top) {
        if (top != -__builtin_inff()) sum *= exp64(((double)top - (double)m) * inv_t);
        top = m;
      }
      const float base = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
      for (int k = 0; k < UNR; ++k) {
        float e[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) e[i] = __builtin_amdgcn_exp2f((f[k][i] - base) * c);
        sum += (double)(((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])));
      }
    }
  }
  // over the workgroup
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float mine = top;
  top = wave_max(top);
  if (temp == 0.0f) {
    at = mine == top ? at : 0x7FFFFFFF;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
      const int other = __shfl_xor(at, x);
      at = other < at ? other : at;
    }
  } else if (mine != top && mine != -__builtin_inff()) {
    sum *= exp64(((double)mine - (double)top) / (double)temp);
  }
  sum = sum64(sum);
  if (lane == 0) {
    s_top[wave] = top;
    s_at[wave] = at;
    s_sum[wave] = sum;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 4; ++w) best(top, at, s_top[w], s_at[w]);
    sum = 0.0;
    for (int w = 0; w < 4; ++w)
      sum += s_top[w] == top || s_top[w] == -__builtin_inff() || temp == 0.0f
                 ? s_sum[w] : s_sum[w] * exp64(((double)s_top[w] - (double)top) / (double)temp);
    RowStat* const st = a.stats + (size_t)t * a.splits + split;
    store_agent(&st->top_at, (uint64_t)(uint32_t)at << 32 | __float_as_uint(top));
    store_agent(&st->sum, sum);
    if (split == 0) {
      store_agent(&a.row_drafts[t].logit_id, (uint64_t)(uint32_t)d.x << 32 | __float_as_uint(d.l));
      store_agent(&a.row_drafts[t].uq, d.uq);
    }
  }
  if (!last_of(counter_of(a, r), (uint32_t)(sp.n * a.splits), &s_last)) return;
  const Choice c = choose<T, Q, false>(a, r, sp, before, temp, sh);
  if (threadIdx.x == 0) a.choices[r] = c;
  put_rows(a, c, r);
}

// ---------------------------------------------------------------- B: the row that is drawn from

// eight weights from j on; 0 past the end
template <class T, class Q, bool PROBS>
__device__ __forceinline__ void weights(const DraftArgs& a, const Choice& c, int j, double inv_z, bool plain, double* w) {
  float f[kVec];
  load_row((const T*)a.target + (int64_t)(c.t0 + c.count) * a.t_stride, j, a.vocab, PROBS ? 0.0f : -__builtin_inff(), f);
  float q[kVec];
  const bool less = !plain && c.q_row >= 0;
  if (less) load_row((const Q*)a.draft + c.q_row * a.d_stride, j, a.vocab, 0.0f, q);
#pragma unroll
  for (int i = 0; i < kVec; ++i) w[i] = PROBS ? (double)f[i] : exp64(((double)f[i] - c.top) * c.inv_t) * inv_z;
  if (less) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const double d = w[i] - (double)q[i];
      w[i] = d > 0.0 ? d : d == d ? 0.0 : d;      // NaN stays
    }
  }
  if (!plain && c.without >= j && c.without < j + kVec)
#pragma unroll
    for (int i = 0; i < kVec; ++i) w[i] = j + i == c.without ? 0.0 : w[i];
}

__device__ __forceinline__ double block_sum(double v, double* s) {
  v = sum64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return s[0] + s[1] + s[2] + s[3];
}

template <class T, class Q, bool PROBS>
__device__ __forceinline__ double chunk_sum(const DraftArgs& a, const Choice& c, int g, double inv_z, bool plain, double* s) {
  const int per = part_size(a.vocab, a.chunks), from = g * per, end = from + per < a.vocab ? from + per : a.vocab;
  double sum = 0.0;
  for (int j = from + threadIdx.x * kVec; j < end; j += kThreads * kVec) {
    double w[kVec];
    weights<T, Q, PROBS>(a, c, j, inv_z, plain, w);
#pragma unroll
    for (int i = 0; i < kVec; ++i) sum += j + i < end ? w[i] : 0.0;
  }
  return block_sum(sum, s);
}

// The place in chunk `g` where the sum that starts at `before` passes t, or the
// last weight that is not 0.
template <class T, class Q, bool PROBS>
__device__ __forceinline__ int place_in(const DraftArgs& a, const Choice& c, int g, double before, double t, double inv_z,
                                        bool plain, double* s, int* s_at) {
  const int per = part_size(a.vocab, a.chunks), from = g * per, end = from + per < a.vocab ? from + per : a.vocab;
  const int wave = threadIdx.x >> 6;
  int last = -1;
  for (int base = from; base < end; base += kThreads * kVec) {
    const int j = base + threadIdx.x * kVec;
    double w[kVec], mine = 0.0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) w[i] = 0.0;
    if (j < end) weights<T, Q, PROBS>(a, c, j, inv_z, plain, w);
    int hit = 0x7FFFFFFF, nonzero = -1;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (j + i >= end) w[i] = 0.0;
      mine += w[i];
      if (w[i] > 0.0) nonzero = j + i;
    }
    const double upto = scan64(mine);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) s[wave] = upto;
    if (threadIdx.x == 0) s_at[0] = 0x7FFFFFFF, s_at[1] = -1;
    __syncthreads();
    double sum = before + (upto - mine);
    for (int x = 0; x < wave; ++x) sum += s[x];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      sum += w[i];
      if (hit == 0x7FFFFFFF && sum > t && w[i] > 0.0) hit = j + i;
    }
    if (hit != 0x7FFFFFFF) atomicMin(&s_at[0], hit);
    if (nonzero >= 0) atomicMax(&s_at[1], nonzero);
    __syncthreads();
    if (s_at[0] != 0x7FFFFFFF) return s_at[0];
    if (s_at[1] >= 0) last = s_at[1];
    before += s[0] + s[1] + s[2] + s[3];
  }
  return last;
}

// The chunk where the sum of the chunks' (one a lane; every wave finds it) passes u
// times all, and the sum before it; -1: nowhere.
struct Found {
  int chunk;
  double before, t;
};
__device__ __forceinline__ Found find_chunk(double mine, float u, bool& none) {
  const double upto = scan64(mine), total = lane64(upto, 63);
  Found f{-1, 0.0, (double)u * total};
  none = total == 0.0;
  if (!(total > 0.0 && total < __builtin_inf())) return f;
  const uint64_t past = __ballot(upto > f.t), some = __ballot(mine > 0.0);
  f.chunk = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);    // u of 1 or more: the last weight
  f.before = f.chunk ? lane64(upto, f.chunk - 1) : 0.0;
  return f;
}

// What a chunk leaves of a row from which q is subtracted.
struct Sums {
  double e, e_s, q_s, near;
};
constexpr double kNear = 1.0 / 65536, kOff = 1e-10;

template <class T, class Q>
__device__ __forceinline__ Sums chunk_sums(const DraftArgs& a, const Choice& c, int g, double inv_z, double (&s)[4][4]) {
  const int per = part_size(a.vocab, a.chunks), from = g * per, end = from + per < a.vocab ? from + per : a.vocab;
  double v[4] = {0.0, 0.0, 0.0, 0.0};
  for (int j = from + threadIdx.x * kVec; j < end; j += kThreads * kVec) {
    float f[kVec], q[kVec];
    load_row((const T*)a.target + (int64_t)(c.t0 + c.count) * a.t_stride, j, end, -__builtin_inff(), f);
    load_row((const Q*)a.draft + c.q_row * a.d_stride, j, end, 0.0f, q);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const double e = exp64(((double)f[i] - c.top) * c.inv_t), p = e * inv_z, d = p - (double)q[i];
      v[0] += e;
      v[1] += d > 0.0 ? e : 0.0;
      v[2] += d > 0.0 ? (double)q[i] : d == d ? 0.0 : d;     // NaN stays
      v[3] += __builtin_fabs(d) <= kNear * p ? p : 0.0;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = sum64(v[k]);
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k][threadIdx.x >> 6] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = s[k][0] + s[k][1] + s[k][2] + s[k][3];
  return Sums{v[0], v[1], v[2], v[3]};
}

template <class T, class Q, bool PROBS>
__global__ __launch_bounds__(kThreads) void k_next(DraftArgs a) {
  __shared__ ChooseShared sh;
  __shared__ double s[4], s4[4][4], s_part[64];
  __shared__ int s_at[2], s_last;
  const int r = blockIdx.x / a.chunks, g = blockIdx.x % a.chunks, lane = threadIdx.x & 63;
  const Span sp = token_span(a.q_start, r, a.tokens);
  Choice c;
  if constexpr (PROBS) {
    c = choose<T, Q, true>(a, r, sp, a.draft ? draft_rows_before(a, r, sp.t0) : 0, 1.0f, sh);
    if (g == 0) put_rows(a, c, r);
    if (g == 0 && r == a.requests - 1) {                // rows of no request
      const int behind = a.q_start[a.requests];
      for (int t = (behind < 0 ? 0 : behind) + threadIdx.x; t < a.tokens; t += kThreads) a.out[t] = -1;
    }
  } else {
    if (sp.n <= 0) return;
    c = a.choices[r];
    // No workgroup of A has left it where q_start falls or changes, or counters were
    // not 0: what is used as a place stays inside the request all the same.
    c.t0 = sp.t0;
    c.count = c.count < 0 ? 0 : c.count >= sp.n ? sp.n - 1 : c.count;
    c.q_row = a.draft && c.q_row < a.draft_rows ? c.q_row : -1;
  }
  if (!c.draw) return;
  const float u = a.u_next[r];
  Sums* const parts = (Sums*)a.parts + (size_t)r * a.chunks;
  const bool two = !PROBS && c.q_row >= 0;              // Z is still to be found
  if (two) {
    const Sums v = chunk_sums<T, Q>(a, c, g, 1.0 / c.z, s4);
    if (threadIdx.x < 4) store_agent((double*)(parts + g) + threadIdx.x, threadIdx.x == 0 ? v.e : threadIdx.x == 1 ? v.e_s
                                                                         : threadIdx.x == 2 ? v.q_s : v.near);
  } else {
    const double sum = chunk_sum<T, Q, PROBS>(a, c, g, 1.0, false, s);
    if (threadIdx.x == 0) store_agent(&parts[g].e, sum);
  }
  if (!last_of(counter_of(a, r), (uint32_t)a.chunks, &s_last)) return;
  double mine = lane < a.chunks ? load_agent(&parts[lane].e) : 0.0, inv_z = 1.0;
  bool again = false, none = false;
  if (two) {
    const int k = lane < a.chunks ? lane : 0;
    const double e_s = load_agent(&parts[k].e_s), q_s = load_agent(&parts[k].q_s), near = load_agent(&parts[k].near);
    __builtin_amdgcn_sched_barrier(0);                  // (all loads before the first wait)
    inv_z = 1.0 / sum64(mine);
    mine = lane < a.chunks ? e_s * inv_z - q_s : 0.0;
    mine = mine < 0.0 ? 0.0 : mine;
    const double off = __builtin_fabs(c.z * inv_z - 1.0);
    again = off > kNear * 0.5 || off * sum64(lane < a.chunks ? near : 0.0) > kOff * sum64(mine);
  }
  Found f = find_chunk(mine, u, none);
  bool plain = false;
  for (int turn = 0; turn < 2; ++turn) {
    // the chunks' weights with Z, or, where nothing is left of p, of p itself
    if (turn == 0 && !again) continue;
    if (turn == 1) {
      if (!none || (c.q_row < 0 && c.without < 0)) break;
      plain = true;
    }
    for (int k = 0; k < a.chunks; ++k) {
      const double one = chunk_sum<T, Q, PROBS>(a, c, k, inv_z, plain, s);
      if (threadIdx.x == 0) s_part[k] = one;
    }
    __syncthreads();
    f = find_chunk(lane < a.chunks ? s_part[lane] : 0.0, u, none);
    __syncthreads();
  }
  const int next = f.chunk < 0 ? -1 : place_in<T, Q, PROBS>(a, c, f.chunk, f.before, f.t, inv_z, plain, s, s_at);
  if (threadIdx.x == 0) a.out[c.t0 + c.count] = next;
}

template <class T, class Q>
void run(const DraftArgs& a, hipStream_t st) {
  const dim3 block(kThreads), next((unsigned)(a.requests * a.chunks));
  if (a.probs) {
    hipLaunchKernelGGL((k_next<T, Q, true>), next, block, 0, st, a);
    return;
  }
  hipLaunchKernelGGL((k_stats<T, Q>), dim3((unsigned)(a.tokens * a.splits)), block, 0, st, a);
  // (greedy for all: A has found the next tokens; 4 us)
  if (a.temps || a.temp != 0.0f) hipLaunchKernelGGL((k_next<T, Q, false>), next, block, 0, st, a);
}

}  // namespace

// A: about 768 workgroups, none below 4096 elements (208 rows of 131072 in bf16:
// 18.4 us; 2048 workgroups 22.1); a drawn row in chunks of 2048, one load a lane, 64
// at most, and 32 where the requests fill the chip with them (B over 131072 elements,
// us with 64 and 32: 16 requests 13.2 and 15.8, 64 28.5 and 28, 128 55 and 47-50).
DraftPlan draft_plan(int tokens, int requests, int vocab, int probs) {
  DraftPlan p{1, 1, 0, 0, 0, 0};
  const int64_t want = tokens > 0 ? (768 + tokens - 1) / tokens : 1, fit = (vocab + 4095) / 4096;
  p.splits = (int)(want < fit ? want : fit);
  p.splits = p.splits < 1 ? 1 : p.splits > 64 ? 64 : p.splits;
  p.chunks = (vocab + 2047) / 2048;
  const int most = requests > 64 ? 32 : 64;
  p.chunks = p.chunks > most ? most : p.chunks;
  p.drafts_at = probs ? 0 : (size_t)tokens * p.splits * sizeof(RowStat);
  p.choices_at = p.drafts_at + (probs ? 0 : (size_t)tokens * sizeof(RowDraft));
  p.parts_at = p.choices_at + (probs ? 0 : (size_t)requests * sizeof(Choice));
  p.bytes = p.parts_at + (size_t)requests * p.chunks * sizeof(Sums);
  return p;
}

int launch_drafts(const DraftArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (a.t_bf16) {
    if (a.d_bf16) run<uint16_t, uint16_t>(a, st);
    else run<uint16_t, float>(a, st);
  } else {
    if (a.d_bf16) run<float, uint16_t>(a, st);
    else run<float, float>(a, st);
  }
  return (int)hipGetLastError();
}

}  // namespace ocq
