// The next step's tables from what the last one left, on the GPU.
//
// Request r had kv tokens in the cache, n of them new in the last step, of which 1
// + accepted stay; it brings new[r] tokens to the next one (< 0: it has ended and
// keeps nothing).  So
//   kept = kv - n + min(n, 1 + accepted),  kv' = kept + new,
//   need = ceil(kv' / page_size) pages,
// and the pages beyond those it holds come from a ring of free ones, those it no
// longer needs go back there: `taken` and `given` count the entries ever taken out
// and put in, so that what is put in lies behind all that can be taken in the same
// step and every entry's place follows from sums over the requests before.
//
// One workgroup sums over the requests.  A small step (kSmall tokens, one request a
// thread) ends in the same launch: a thread per page that moves and per token,
// its request found in LDS.  A large one hands each request's sums to a second
// launch with workgroups of every request.  Latency bounds it: 16 requests of 13 tokens
// 4.3 us; 2048 requests, 128 of them starting on up to 4096 tokens each, 5.7 and 11
// (their 5 MB: 1).
#include "kcommon.h"
#include "step.h"

namespace ocq {
namespace {

constexpr int kWide = 1024, kSmall = 16384;

struct Rec {
  int start, fresh;          // first token, new tokens
  int kept, held, need, got; // tokens that stay, pages held, needed, in hand at the end
  int take, give;            // first of the ring entries taken, given
};

// Inclusive sums over the lanes (DPP: rows of 16, then across them).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// The place `n` entries behind place `from` of the ring, both below its size (a
// remainder in 64 bits for every token took longer than all else; counts that no step
// leaves give any n).
__device__ __forceinline__ int ring_at(const TableArgs& a, int from, int n) {
  uint32_t at = (uint32_t)from + (uint32_t)n;
  at = at >= (uint32_t)a.ring_size ? at - (uint32_t)a.ring_size : at;
  return at < (uint32_t)a.ring_size ? (int)at : 0;
}

// page j of a request's row after the step, from what was there before it
__device__ __forceinline__ int page_of(const TableArgs& a, const Rec& q, int r, int j, int taken) {
  if (j < 0 || j >= a.max_pages) return -1;
  if (j < q.held) return a.table[r * a.table_stride + j];
  return j < q.got ? a.ring[ring_at(a, taken, q.take + j - q.held)] : -1;
}

// place of a request's new token i (past 2^31: below 0, without a page)
__device__ __forceinline__ int place_of(const Rec& q, int i) { return (int)((unsigned)q.kept + (unsigned)i); }

__device__ __forceinline__ void put_token(const TableArgs& a, const Rec& q, int r, int t, int i, int page) {
  const int place = place_of(q, i);
  if (a.slots) a.slots[t] = page >= 0 ? ((int64_t)page << a.page_shift) + (place & ((1 << a.page_shift) - 1)) : -1;
  if (a.positions) a.positions[t] = place;
  if (a.owners) a.owners[t] = r;
}

__device__ __forceinline__ void no_token(const TableArgs& a, int t) {
  if (a.slots) a.slots[t] = -1;
  if (a.positions) a.positions[t] = -1;
  if (a.owners) a.owners[t] = -1;
}

// (numbers of tokens whose sums pass 2^31 give any j)
__device__ __forceinline__ void take_page(const TableArgs& a, const Rec& q, int r, int j, int taken) {
  if (j < q.held || j >= q.need) return;
  a.table[r * a.table_stride + j] = j < q.got ? a.ring[ring_at(a, taken, q.take + j - q.held)] : -1;
}
__device__ __forceinline__ void give_page(const TableArgs& a, const Rec& q, int r, int j, int given) {
  if (j < q.need || j >= q.held) return;
  a.ring[ring_at(a, given, q.give + j - q.need)] = a.table[r * a.table_stride + j];
}

// the last of n (> 0) sorted numbers that is not above v, the first of them not above it
__device__ __forceinline__ int last_le(const int* s, int n, int v) {
  int lo = 0;
  for (int step = 512; step > 0; step >>= 1)
    if (lo + step < n && s[lo + step] <= v) lo += step;
  return lo;
}

template <bool SMALL>
__global__ __launch_bounds__(kWide) void k_sums(TableArgs a) {
  __shared__ int s_sum[3][16], s_prev;
  __shared__ unsigned long long s_over;
  __shared__ int s_start[SMALL ? kWide : 1], s_take[SMALL ? kWide : 1], s_give[SMALL ? kWide : 1];
  __shared__ Rec s_rec[SMALL ? kWide : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t taken = (uint64_t)a.counts_in[0], given = (uint64_t)a.counts_in[1];
  const uint64_t span = given - taken, size = (uint64_t)a.ring_size;
  const int from = (int)(taken % size), to = (int)(given % size);   // where entries come from and go to
  const int free = (int64_t)span < 0 ? 0 : span > (uint64_t)a.ring_size ? a.ring_size : (int)span;
  int c_new = 0, c_want = 0, c_back = 0;
  int64_t over = 0;
  if (threadIdx.x == 0) s_over = 0;
  for (int base = 0; base < a.requests; base += kWide) {
    const int r = base + threadIdx.x;
    const bool in = r < a.requests;
    int q0 = 0, q1 = 0, kv = 0, held = 0, fresh = 0, acc = 0x7FFFFFFE;
    if (in) {
      // (outputs may be the inputs: the entry before this tile's first was kept)
      q0 = base > 0 && threadIdx.x == 0 ? s_prev : a.q_in[r];
      q1 = a.q_in[r + 1];
      kv = a.kv_in[r];
      held = a.held_in[r];
      fresh = a.news[r];
      if (a.accepted) acc = a.accepted[r];
    }
    __syncthreads();
    if (threadIdx.x == kWide - 1) s_prev = q1;
    const int n = q1 > q0 ? q1 - q0 : 0;
    acc = acc < -1 ? -1 : acc;
    int64_t kept = (int64_t)kv - n + (acc < n ? acc + 1 < n ? acc + 1 : n : n);
    kept = kept < 0 || fresh < 0 ? 0 : kept;
    fresh = fresh < 0 ? 0 : fresh;
    const int64_t most = 0x7FFFFFFF;
    const int64_t kv_out = kept + fresh < most ? kept + fresh : most;
    const int64_t pages = (kv_out + (1 << a.page_shift) - 1) >> a.page_shift;
    held = held < 0 ? 0 : held > a.max_pages ? a.max_pages : held;
    const int need = pages < a.max_pages ? (int)pages : a.max_pages;
    const int want = need > held ? need - held : 0, back = held > need ? held - need : 0;
    int v[3] = {in ? fresh : 0, in ? want : 0, in ? back : 0}, sum[3];
    if (in) over += pages - need;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      sum[k] = wave_scan(v[k]);
      if (lane == 63) s_sum[k][wave] = sum[k];
    }
    __syncthreads();
    int all[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int w = lane < 16 ? s_sum[k][lane] : 0, upto = wave_scan(w);
      sum[k] += wave > 0 ? __builtin_amdgcn_readlane(upto, wave - 1) : 0;
      all[k] = __builtin_amdgcn_readlane(upto, 15);
    }
    const int start = c_new + sum[0] - v[0], take = c_want + sum[1] - v[1], give = c_back + sum[2] - v[2];
    if (in) {
      const int left = free - take < 0 ? 0 : free - take, got = want < left ? want : left;
      const Rec rec{start, fresh, (int)kept, held, need, need > held ? held + got : need, take, give};
      a.q_out[r + 1] = start + fresh;
      if (r == 0) a.q_out[0] = 0;
      a.kv_out[r] = (int)kv_out;
      a.held_out[r] = rec.got;
      if constexpr (SMALL) {
        s_start[r] = start;
        s_take[r] = take;
        s_give[r] = give;
        s_rec[r] = rec;
      } else {
        ((Rec*)a.records)[1 + r] = rec;
      }
    }
    c_new += all[0];
    c_want += all[1];
    c_back += all[2];
    __syncthreads();
  }
  // pages beyond the table's rows are missing as well (few requests have any; all of
  // them may be more than an int holds)
  if (over) atomicAdd(&s_over, (unsigned long long)over);
  __syncthreads();
  if (threadIdx.x == 0) {
    const int64_t missing = (int64_t)s_over + (c_want > free ? c_want - free : 0);
    if (a.missing) a.missing[0] = missing < 0x7FFFFFFF ? (int)missing : 0x7FFFFFFF;
    a.counts_out[0] = (int64_t)(taken + (uint64_t)(c_want < free ? c_want : free));
    a.counts_out[1] = (int64_t)(given + (uint64_t)c_back);
    if constexpr (!SMALL) {
      a.records[0] = from;
      a.records[1] = to;
      a.records[2] = c_new;
    }
  }
  if constexpr (SMALL) {
    const int n = a.requests;
    // tokens and pages read the table's old entries and the ring's free ones; what
    // is written lies elsewhere
    for (int t = threadIdx.x; t < a.tokens; t += kWide) {
      if (t >= c_new) {
        no_token(a, t);
        continue;
      }
      const int r = last_le(s_start, n, t);
      const Rec& q = s_rec[r];
      const int i = t - q.start;
      put_token(a, q, r, t, i, a.slots ? page_of(a, q, r, place_of(q, i) >> a.page_shift, from) : -1);
    }
    for (int i = threadIdx.x; i < c_want; i += kWide) {
      const int r = last_le(s_take, n, i);
      take_page(a, s_rec[r], r, s_rec[r].held + i - s_take[r], from);
    }
    for (int i = threadIdx.x; i < c_back; i += kWide) {
      const int r = last_le(s_give, n, i);
      give_page(a, s_rec[r], r, s_rec[r].need + i - s_give[r], to);
    }
  }
}

// A request's pages and tokens; grid.y workgroups share them.
__global__ __launch_bounds__(256) void k_fill(TableArgs a) {
  const int r = blockIdx.x, first = blockIdx.y * 256 + threadIdx.x, step = gridDim.y * 256;
  const int taken = a.records[0], given = a.records[1];
  const Rec q = ((const Rec*)a.records)[1 + r];
  if (q.start >= 0) {
    // four tokens of a lane at a time: their pages are on their way together
    const int n = q.fresh < a.tokens - q.start ? q.fresh : a.tokens - q.start;
    for (int i0 = first; i0 < n; i0 += 4 * step) {
      int page[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * step;
        page[k] = a.slots && i < n ? page_of(a, q, r, place_of(q, i) >> a.page_shift, taken) : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i0 + k * step < n) put_token(a, q, r, q.start + i0 + k * step, i0 + k * step, page[k]);
    }
  }
  for (int j = q.held + first; j < q.need; j += step) take_page(a, q, r, j, taken);
  for (int j = q.need + first; j < q.held; j += step) give_page(a, q, r, j, given);
  if (r == a.requests - 1)
    for (int t = (a.records[2] < 0 ? 0 : a.records[2]) + first; t < a.tokens; t += step) no_token(a, t);
}

// (one workgroup moves every page of a small step: all of 2^19 at once take 0.35 ms)
bool small(int requests, int tokens, int max_pages) {
  return requests <= kWide && tokens <= kSmall && (int64_t)requests * max_pages <= 1 << 19;
}

}  // namespace

size_t table_workspace(int requests, int tokens, int max_pages) {
  return small(requests, tokens, max_pages) ? 0 : ((size_t)requests + 1) * sizeof(Rec);
}

int launch_tables(const TableArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (small(a.requests, a.tokens, a.max_pages)) {
    hipLaunchKernelGGL((k_sums<true>), dim3(1), dim3(kWide), 0, st, a);
    return (int)hipGetLastError();
  }
  hipLaunchKernelGGL((k_sums<false>), dim3(1), dim3(kWide), 0, st, a);
  // (2048 requests, 128 of them starting on 4096 tokens: 13.0 us, twice as many
  // workgroups 11.0)
  int y = 2 * (a.tokens / (a.requests * 256) + 1);
  y = y > 64 ? 64 : y;
  hipLaunchKernelGGL(k_fill, dim3((unsigned)a.requests, (unsigned)y), dim3(256), 0, st, a);
  return (int)hipGetLastError();
}

}  // namespace ocq
