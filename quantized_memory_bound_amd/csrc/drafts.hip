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
// Three launches.  A reads all logits once: each row's maximum and sum in 32 bits.
// The acceptances compare 64-bit exponentials with that sum, whose relative error
// is below 2^-22.  B sums the drawn row's exponentials in 64 bits (its weights
// subtract q from p, and the place that a random number falls on hangs on every
// weight before it), C its weights, in chunks; the workgroup that ends a request's
// last chunk finds the chunk and the place in it.  Without q the weights need no Z
// and B falls away; with given probabilities A does too.
#include "kcommon.h"
#include "layer_index.h"
#include "step.h"

namespace ocq {

// A part of a row: its maximum, where it first stands, sum of exp((l - max) / T);
// where not every logit is a number, the sum is NaN.
struct RowStat {
  float top;
  int at;
  double sum;
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

// ---------------------------------------------------------------- A: statistics of every row

template <class T>
__global__ __launch_bounds__(kThreads) void k_stats(DraftArgs a) {
  const int t = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int r = request_of(a, t);
  if (r < 0) return;
  const float temp = temperature(a, r);
  const int per = ((a.vocab + a.splits - 1) / a.splits + kVec - 1) / kVec * kVec;
  const int from = split * per, end = from + per < a.vocab ? from + per : a.vocab;
  const T* const row = (const T*)a.target + t * a.t_stride;
  float top = -__builtin_inff();
  int at = 0x7FFFFFFF;
  double sum = 0.0;
  bool bad = false;
  if (temp == 0.0f) {
    for (int j = from + threadIdx.x * kVec; j < end; j += kThreads * kVec) {
      float f[kVec];
      load_row(row, j, end, -__builtin_inff(), f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        bad |= f[i] != f[i];
        if (f[i] > top) {
          top = f[i];
          at = j + i;
        }
      }
    }
  } else {
    const float c = (float)(kLog2e / (double)temp);
    float s = 0.0f;
    for (int j = from + threadIdx.x * kVec; j < end; j += kThreads * kVec) {
      float f[kVec], m = top;
      load_row(row, j, end, -__builtin_inff(), f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) m = fmaxf(m, f[i]);
      if (m > top) {
        s = top == -__builtin_inff() ? s : s * __builtin_amdgcn_exp2f((top - m) * c);
        top = m;
      }
      const float base = top == -__builtin_inff() ? 0.0f : top;
      float e = 0.0f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) e += __builtin_amdgcn_exp2f((f[i] - base) * c);
      s += e;
    }
    sum = s;
  }
  // over the workgroup
  __shared__ float s_top[4];
  __shared__ int s_at[4];
  __shared__ double s_sum[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float mine = top;
  if (bad) sum = __builtin_nan("");
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) best(top, at, __shfl_xor(top, x), __shfl_xor(at, x));
  if (temp != 0.0f && mine != top)
    sum = mine == -__builtin_inff() ? sum : sum * (double)__builtin_amdgcn_exp2f((mine - top) * (float)(kLog2e / temp));
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
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
                 ? s_sum[w] : s_sum[w] * exp(((double)s_top[w] - (double)top) / (double)temp);
    a.stats[(size_t)t * a.splits + split] = RowStat{top, at, sum};
  }
}

// ---------------------------------------------------------------- B, C: the row that is drawn from

// What every workgroup of a request finds out by itself.
struct Choice {
  int t0, n, count;          // first row, rows, accepted drafts
  int greedy, at;            // T = 0: the next token (-1: none)
  double top, inv_t, z;      // of the drawn row (logits)
  int64_t q_row;             // the draft's row that is subtracted, -1: none
  int without;               // the id that is left out, -1: none
};

template <class T, class Q>
__device__ __forceinline__ void choose(const DraftArgs& a, int r, Choice* sh) {
  const Span sp = token_span(a.q_start, r, a.tokens);
  const int n = sp.n < 0 ? 0 : sp.n, lane = threadIdx.x & 63;
  if (threadIdx.x >= 64) return;
  // rows of the draft's before this request's: one less than its tokens each
  int64_t before = 0;
  if (a.draft) {
    int idle = 0;
    for (int base = 0; base < r; base += 64)
      idle += __popcll(__ballot(base + lane < r && token_span(a.q_start, base + lane, a.tokens).n <= 0));
    before = sp.t0 - (r - idle);
  }
  const float temp = a.probs ? 1.0f : temperature(a, r);
  const double inv_t = 1.0 / (double)temp;
  int count = n - 1;
  Choice c{sp.t0, n, 0, 0, -1, 0.0, inv_t, 1.0, -1, -1};
  // a lane's row t: what it says about its draft, and what drawing from it takes
  for (int i0 = 0; i0 < n; i0 += 64) {
    const int i = i0 + lane, t = sp.t0 + (i < n ? i : 0);
    float top = -__builtin_inff();
    int at = 0x7FFFFFFF;
    double z = 0.0;
    if (!a.probs) {
      const RowStat* const st = a.stats + (size_t)t * a.splits;
      for (int k = 0; k < a.splits; ++k) best(top, at, st[k].top, st[k].at);
      for (int k = 0; k < a.splits; ++k)
        z += st[k].top == top || st[k].top == -__builtin_inff() || temp == 0.0f
                 ? st[k].sum : st[k].sum * exp(((double)st[k].top - (double)top) * inv_t);
    }
    bool keep = false;
    if (i < n - 1) {
      const int x = a.ids[t + 1];
      if (x >= 0 && x < a.vocab) {
        double q = 1.0;
        if (a.draft) q = before + i >= 0 && before + i < a.draft_rows
                             ? (double)load1((const Q*)a.draft + (before + i) * a.d_stride + x) : __builtin_nan("");
        const double l = (double)load1((const T*)a.target + t * a.t_stride + x);
        const double u = (double)a.u_accept[t];
        if (a.probs) keep = u * q < l;
        else if (temp == 0.0f) keep = z == 0.0 && u * q < (x == at ? 1.0 : 0.0);
        else keep = u * q * z < exp((l - (double)top) * inv_t);
      }
    }
    const uint64_t out = ~__ballot(keep);
    const int first = i0 + __builtin_ctzll(out);   // (a row past the last draft keeps nothing)
    if (out != 0 && first < n) {
      const int l = first - i0;
      count = first;
      c.top = (double)__shfl(top, l);
      c.z = __shfl(z, l);
      c.at = __shfl(at, l);
      break;
    }
  }
  if (lane != 0) return;
  c.count = n > 0 ? count : 0;
  c.greedy = !a.probs && temp == 0.0f;
  if (!c.greedy || c.at == 0x7FFFFFFF || c.z != 0.0) c.at = -1;
  if (n > 0 && count < n - 1) {
    const int x = a.ids[sp.t0 + count + 1];
    if (a.draft) c.q_row = before + count >= 0 && before + count < a.draft_rows ? before + count : -1;
    else if (x >= 0 && x < a.vocab) c.without = x;
  }
  *sh = c;
}

// eight weights from j on; 0 past the end
template <class T, class Q, bool PROBS>
__device__ __forceinline__ void weights(const DraftArgs& a, const Choice& c, int j, double inv_z, bool plain, double* w) {
  float f[kVec];
  load_row((const T*)a.target + (int64_t)(c.t0 + c.count) * a.t_stride, j, a.vocab, PROBS ? 0.0f : -__builtin_inff(), f);
#pragma unroll
  for (int i = 0; i < kVec; ++i) w[i] = PROBS ? (double)f[i] : exp(((double)f[i] - c.top) * c.inv_t) * inv_z;
  if (plain) return;
  if (c.q_row >= 0) {
    float q[kVec];
    load_row((const Q*)a.draft + c.q_row * a.d_stride, j, a.vocab, 0.0f, q);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const double d = w[i] - (double)q[i];
      w[i] = d > 0.0 ? d : d == d ? 0.0 : d;      // NaN stays
    }
  }
  if (c.without >= j && c.without < j + kVec)
#pragma unroll
    for (int i = 0; i < kVec; ++i) w[i] = j + i == c.without ? 0.0 : w[i];
}

// Sums over the lanes before and with this one.
__device__ __forceinline__ double scan64(double v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const double o = __shfl_up(v, x);
    if (lane >= x) v += o;
  }
  return v;
}

__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) v += __shfl_xor(v, x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return s[0] + s[1] + s[2] + s[3];
}

__device__ __forceinline__ int chunk_size(const DraftArgs& a) {
  return ((a.vocab + a.chunks - 1) / a.chunks + kVec - 1) / kVec * kVec;
}

// The place in chunk `g` where the sum that starts at `before` passes t, or the
// last weight that is not 0.
template <class T, class Q, bool PROBS>
__device__ __forceinline__ int place_in(const DraftArgs& a, const Choice& c, int g, double before, double t, double inv_z,
                                        bool plain, double* s, int* s_at) {
  const int per = chunk_size(a), from = g * per, end = from + per < a.vocab ? from + per : a.vocab;
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

// Z: sums of the exponentials (a launch of its own before the weights'); else the
// sums of the weights, and the next token.
template <class T, class Q, bool PROBS, bool Z>
__global__ __launch_bounds__(kThreads) void k_next(DraftArgs a) {
  __shared__ Choice sh;
  __shared__ double s[4], s_part[64];
  __shared__ int s_at[2], s_last;
  const int r = blockIdx.x / a.chunks, g = blockIdx.x % a.chunks;
  choose<T, Q>(a, r, &sh);
  __syncthreads();
  const Choice c = sh;
  const size_t pairs = (size_t)a.requests * a.chunks;
  double* const parts = a.parts + (Z ? 0 : pairs) + (size_t)r * a.chunks;
  int next = c.at;
  if (c.n > 0 && !c.greedy) {
    const int per = chunk_size(a), from = g * per, end = from + per < a.vocab ? from + per : a.vocab;
    double z = 1.0;
    if (!Z && !PROBS && c.q_row >= 0) {
      z = 0.0;
      for (int k = 0; k < a.chunks; ++k) z += a.parts[(size_t)r * a.chunks + k];
    }
    const double inv_z = 1.0 / z;
    double sum = 0.0;
    if (!Z || c.q_row >= 0)
      for (int j = from + threadIdx.x * kVec; j < end; j += kThreads * kVec) {
        double w[kVec];
        weights<T, Q, PROBS>(a, c, j, inv_z, Z, w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) sum += j + i < end ? w[i] : 0.0;
      }
    sum = block_sum(sum, s);
    if (threadIdx.x == 0) {
      if (Z) parts[g] = sum;
      else __hip_atomic_store((uint64_t*)parts + g, __builtin_bit_cast(uint64_t, sum), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (Z) return;
    // the workgroup that ends the request's last chunk
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (threadIdx.x == 0) {
      const uint32_t before = __hip_atomic_fetch_add(a.counters + r, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s_last = before + 1 == (uint32_t)a.chunks;
      if (s_last) __hip_atomic_store(a.counters + r, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s_last) return;
    for (int plain = 0; plain < 2; ++plain) {
      if (plain && c.q_row < 0 && c.without < 0) break;
      if (threadIdx.x < a.chunks && !plain)
        s_part[threadIdx.x] = __builtin_bit_cast(double, __hip_atomic_load((uint64_t*)parts + threadIdx.x, __ATOMIC_RELAXED,
                                                                           __HIP_MEMORY_SCOPE_AGENT));
      if (plain) {
        // nothing is left of p after q: drawn from p (chunks summed again, here)
        for (int k = 0; k < a.chunks; ++k) {
          double one = 0.0;
          for (int j = k * per + threadIdx.x * kVec; j < k * per + per && j < a.vocab; j += kThreads * kVec) {
            double w[kVec];
            weights<T, Q, PROBS>(a, c, j, inv_z, true, w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) one += j + i < k * per + per && j + i < a.vocab ? w[i] : 0.0;
          }
          one = block_sum(one, s);
          if (threadIdx.x == 0) s_part[k] = one;
        }
      }
      __syncthreads();
      double total = 0.0;
      for (int k = 0; k < a.chunks; ++k) total += s_part[k];
      if (total == 0.0 && !plain) continue;
      next = -1;
      if (total > 0.0 && total < __builtin_inf()) {
        const double t = (double)a.u_next[r] * total;
        double before = 0.0, at_before = 0.0, run = 0.0;
        int chunk = -1;
        for (int k = 0; k < a.chunks; ++k) {
          run += s_part[k];
          if (chunk < 0 && run > t) {
            chunk = k;
            at_before = before;
          }
          before = run;
        }
        if (chunk < 0) {                              // u of 1 or more: the last weight
          for (int k = 0; k < a.chunks; ++k)
            if (s_part[k] > 0.0) chunk = k;
        }
        next = place_in<T, Q, PROBS>(a, c, chunk, at_before, t, inv_z, plain, s, s_at);
      }
      break;
    }
  } else if (Z || g != 0) {
    return;
  }
  // a request's rows: the accepted drafts, the next token, -1
  for (int i = threadIdx.x; i < c.n; i += kThreads)
    a.out[c.t0 + i] = i < c.count ? a.ids[c.t0 + i + 1] : i == c.count ? next : -1;
  if (threadIdx.x == 0) a.accepted[r] = c.count;
  if (r == a.requests - 1) {                          // rows of no request
    int behind = a.q_start[a.requests];
    behind = behind < 0 ? 0 : behind;
    for (int t = behind + threadIdx.x; t < a.tokens; t += kThreads) a.out[t] = -1;
  }
}

template <class T, class Q>
void run(const DraftArgs& a, hipStream_t st) {
  const dim3 block(kThreads), next((unsigned)(a.requests * a.chunks));
  if (a.probs) {
    hipLaunchKernelGGL((k_next<T, Q, true, false>), next, block, 0, st, a);
    return;
  }
  hipLaunchKernelGGL((k_stats<T>), dim3((unsigned)(a.tokens * a.splits)), block, 0, st, a);
  if (a.draft) hipLaunchKernelGGL((k_next<T, Q, false, true>), next, block, 0, st, a);
  hipLaunchKernelGGL((k_next<T, Q, false, false>), next, block, 0, st, a);
}

}  // namespace

DraftPlan draft_plan(int tokens, int requests, int vocab, int probs) {
  DraftPlan p{1, 1, 0, 0};
  auto ways = [&](int64_t rows, int least, int most) {
    int64_t w = (2048 + rows - 1) / rows;
    const int64_t fit = (vocab + least - 1) / least;
    w = w < fit ? w : fit;
    return (int)(w < 1 ? 1 : w > most ? most : w);
  };
  p.splits = ways(tokens > 0 ? tokens : 1, 4096, 64);
  p.chunks = ways(requests > 0 ? requests : 1, 4096, 64);
  p.stats_bytes = probs ? 0 : (size_t)tokens * p.splits * sizeof(RowStat);
  p.bytes = p.stats_bytes + (size_t)2 * requests * p.chunks * sizeof(double);
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
