// Residual addition, RMSNorm and per-token E4M3 quantization in one pass.
//
//   h = x + residual (fp32), residual_out = bf16(h)
//   y = h / sqrt(mean(h^2) + eps) * weight (fp32)
//   codes = E4M3(fl32(y / s)), s = fl32(max|y| / 448), and / or bf16(y)
//
// The norm is taken of the fp32 sum, not of its bf16 rounding: each output is
// rounded once.  WPR waves hold one row in registers (8 values per lane and
// unit), so x and the residual are read once; two reductions (sum of squares,
// then max|y|) meet in LDS.  WPR is the smallest that keeps a lane at one or two
// units (16 waves from 8192 values on), so that a row's loads are in flight at
// once.  Bound by HBM: 8191 x 4096 rows, both outputs (302 MB), 52 us by the
// kernel trace over three inputs in turn, 57 us a pass where neither inputs nor
// outputs are in the memory-side cache (5.3 TB/s; a device copy runs at 4.7); 208 x
// 4096 rows 5.4 us and one row 2.8 us by latency (load, two reductions, store),
// against 1.6 us for an empty launch.
#include "layer_dev.h"

namespace ocq {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

template <int WPR, int PER, bool PASS>
__global__ __launch_bounds__(WPR < 4 ? 256 : 64 * WPR) void k_norm(NormArgs a) {
  constexpr int RPB = WPR < 4 ? 4 / WPR : 1;   // rows per workgroup
  __shared__ float s_sum[RPB][WPR], s_max[RPB][WPR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int slot = wave / WPR, wr = wave % WPR;
  const int row = blockIdx.x * RPB + slot;
  const bool live = row < a.rows;
  const int units = a.hidden / 8;
  constexpr bool kHoldW = PER <= 2;            // longer rows read the weight again rather than spill
  float h[PER][8];
  v4i w[kHoldW ? PER : 1];
  auto load = [&](const uint16_t* p) { return PASS ? ld_nt((const v4i*)p) : *(const v4i*)p; };
  float ss = 0.0f;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int u = (p * WPR + wr) * 64 + lane;
    const bool in = live && u < units;
    const v4i xv = in ? load(a.x + row * a.x_stride + u * 8) : v4i{0, 0, 0, 0};
    const v4i rv = in && a.res ? load(a.res + row * a.res_stride + u * 8) : v4i{0, 0, 0, 0};
    if constexpr (kHoldW) w[p] = in ? *(const v4i*)(a.w + u * 8) : v4i{0, 0, 0, 0};
    float r[8];
    unpack8_bf16(xv, h[p]);
    unpack8_bf16(rv, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[p][j] += r[j];
      ss = __builtin_fmaf(h[p][j], h[p][j], ss);
    }
    if (in && a.res_out)
      *(v4i*)(a.res_out + (size_t)row * a.hidden + u * 8) =
          pack8_bf16(h[p]);
  }
  ss = wave_sum(ss);
  if constexpr (WPR > 1) {
    if (lane == 0) s_sum[slot][wr] = ss;
    lds_barrier();
    ss = 0.0f;
#pragma unroll
    for (int k = 0; k < WPR; ++k) ss += s_sum[slot][k];
  }
  const float inv = 1.0f / __builtin_sqrtf(ss / (float)a.hidden + a.eps);
  float amax = 0.0f;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int u = (p * WPR + wr) * 64 + lane;
    if constexpr (!kHoldW) w[0] = u < units ? *(const v4i*)(a.w + u * 8) : v4i{0, 0, 0, 0};
    float wf[8];
    unpack8_bf16(w[kHoldW ? p : 0], wf);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[p][j] = h[p][j] * inv * wf[j];
      amax = max_mag(amax, h[p][j]);
    }
    if (live && u < units && a.y)
      *(v4i*)(a.y + (size_t)row * a.hidden + u * 8) =
          pack8_bf16(h[p]);
  }
  if (!a.codes) return;
  if (a.eps == 0.0f && ss == 0.0f) {
    // 0 / 0 in every place of a zero row, whose codes are 0 all the same; what is
    // not zero here is infinite
    amax = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(h[p][j]));
  }
  amax = wave_max(amax < __builtin_inff() ? amax : __builtin_inff());   // NaN as infinity, which fmaxf keeps
  if constexpr (WPR > 1) {
    if (lane == 0) s_max[slot][wr] = amax;
    lds_barrier();
#pragma unroll
    for (int k = 0; k < WPR; ++k) amax = fmaxf(amax, s_max[slot][k]);
  }
  // a row whose squares do not sum to a finite number has no norm: its scale
  // says so, as it does for a y that is not finite
  const float s = ss < __builtin_inff() ? e4m3_scale(amax) : __builtin_nanf("");
  const Quot qt = e4m3_quot_of(s, h);
  if (!live) return;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int u = (p * WPR + wr) * 64 + lane;
    if (u < units) {
      const v2u c = s > 0.0f ? e4m3x8_quot(h[p], qt.s, qt.rcp) : v2u{0u, 0u};
      *(v2u*)(a.codes + (size_t)row * a.hidden + u * 8) = c;
    }
  }
  if (wr == 0 && lane == 0) a.scales[row] = s;
}

template <int WPR, int PER>
int run(const NormArgs& all, hipStream_t st) {
  constexpr int RPB = WPR < 4 ? 4 / WPR : 1;
  constexpr int threads = WPR < 4 ? 256 : 64 * WPR;
  constexpr int at_once = kLanesAtOnce / (64 * WPR);   // a multiple of RPB
  // Inputs far larger than the L2s pass through them without staying (8191 x 4096
  // rows: 55.9 -> 51.8 us by the kernel trace, 61.0 -> 56.5 a pass over cold
  // memory); smaller ones are best kept (2048 x 4096: 15.6 and 15.1).
  const bool pass = (int64_t)all.rows * all.hidden > (1 << 24);
  NormArgs a = all;
  for (int64_t done = 0; done < all.rows; done += at_once) {
    a.rows = all.rows - done < at_once ? (int)(all.rows - done) : at_once;
    const dim3 grid((a.rows + RPB - 1) / RPB);
    if (pass) hipLaunchKernelGGL((k_norm<WPR, PER, true>), grid, dim3(threads), 0, st, a);
    else hipLaunchKernelGGL((k_norm<WPR, PER, false>), grid, dim3(threads), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    const int64_t out = (int64_t)at_once * a.hidden;
    a.x += at_once * a.x_stride;
    if (a.res) a.res += at_once * a.res_stride;
    if (a.res_out) a.res_out += out;
    if (a.y) a.y += out;
    if (a.codes) a.codes += out;
    if (a.scales) a.scales += at_once;
  }
  return 0;
}

}  // namespace

int launch_norm(const NormArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int waves = (a.hidden / 8 + 63) / 64;   // 64-lane units of a row
  if (waves <= 1) return run<1, 1>(a, st);
  if (waves <= 4) return run<4, 1>(a, st);
  if (waves <= 8) return run<4, 2>(a, st);
  if (waves <= 16) return run<16, 1>(a, st);
  if (waves <= 32) return run<16, 2>(a, st);
  if (waves <= 64) return run<16, 4>(a, st);
  return run<16, 8>(a, st);
}

}  // namespace ocq
