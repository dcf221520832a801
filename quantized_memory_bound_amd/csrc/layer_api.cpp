// C-ABI entry points of the operators around the MLP block: argument checks,
// rotary frequencies, launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>

#include "layer.h"
#include "ocq_internal.h"

using namespace ocq;

namespace {

ocq_status hip_error(int rc) {
  char buf[256];
  std::snprintf(buf, sizeof(buf), "kernel launch: %s (%d)", hipGetErrorString((hipError_t)rc), rc);
  return set_error(OCQ_ERR_DEVICE, buf);
}

ocq_status invalid(const char* msg) { return set_error(OCQ_ERR_INVALID_ARG, msg); }
ocq_status unsupported(const char* msg) { return set_error(OCQ_ERR_UNSUPPORTED, msg); }

bool aligned(const void* p, uintptr_t n = 16) { return ((uintptr_t)p & (n - 1)) == 0; }

// strides that keep every byte offset far from 2^63, and 16-byte aligned in units of `per16` elements
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxPage = 0xFFFFFFFFll, kMaxInPage = 0x7FFFFFFFll, kMaxScaleInPage = 0x3FFFFFFFll;
bool stride_ok(int64_t s, int per16) { return s >= 0 && s <= kMaxStride && s % per16 == 0; }

ocq_status check_cache(const ocq_kv_cache* c) {
  if (!c) return invalid("cache is null");
  if (c->format != OCQ_CACHE_BF16 && c->format != OCQ_CACHE_E4M3) return invalid("cache format must be 0 or 1");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return unsupported("head_dim must be 64, 128 or 256");
  if (c->page_size < 1 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return unsupported("page_size must be a power of two in [1, 1024]");
  if (c->num_pages < 1 || c->kv_heads < 1 || c->kv_heads > 4096)
    return invalid("num_pages and kv_heads (up to 4096) must be positive");
  if (!c->k_dev || !c->v_dev) return invalid("null cache pointer");
  if (!aligned(c->k_dev) || !aligned(c->v_dev)) return invalid("cache pointers must be 16-byte aligned");
  const int per16 = c->format == OCQ_CACHE_E4M3 ? 16 : 8;
  if (!stride_ok(c->page_stride, per16) || !stride_ok(c->head_stride, per16) || !stride_ok(c->token_stride, per16))
    return invalid("cache strides must be multiples of 16 bytes, not negative");
  const int64_t esz = 16 / per16;
  if (c->page_stride * esz > kMaxPage || (c->page_size - 1) * c->token_stride * esz > kMaxInPage)
    return unsupported("page strides must be below 2^32 bytes, a page's rows within 2^31");
  if (c->format == OCQ_CACHE_E4M3) {
    if (!c->k_scale_dev || !c->v_scale_dev) return invalid("an E4M3 cache needs scales");
    if (!aligned(c->k_scale_dev, 4) || !aligned(c->v_scale_dev, 4)) return invalid("misaligned scale pointer");
    if (!stride_ok(c->scale_page_stride, 1) || !stride_ok(c->scale_head_stride, 1) ||
        !stride_ok(c->scale_token_stride, 1))
      return invalid("scale strides must not be negative");
    // (attention holds a scale's byte offset in its page in 32 bits; in 64 a verify
    // pass of 16 x 13 tokens over 512 E4M3 keys takes 18.0 us instead of 17.6)
    if (c->scale_page_stride > kMaxPage || (c->page_size - 1) * c->scale_token_stride > kMaxScaleInPage)
      return unsupported("scale page strides must be below 2^32, a page's rows within 2^30");
  }
  return OCQ_OK;
}

ocq_status check_batch(const ocq_token_batch* b, const ocq_kv_cache* c, int heads) {
  if (!b) return invalid("batch is null");
  if (b->requests < 0 || b->tokens < 0) return invalid("requests and tokens must not be negative");
  if (heads < 1 || heads > 65536 || heads % c->kv_heads) return invalid("heads must be a multiple of kv_heads, up to 65536");
  if ((int64_t)b->tokens * heads >= (int64_t)1 << 31) return unsupported("tokens * heads must be below 2^31");
  if (b->requests == 0 || b->tokens == 0) return OCQ_OK;
  if (b->requests > 65536) return unsupported("at most 65536 requests");
  if (b->max_pages < 1 || (int64_t)b->max_pages * c->page_size >= (int64_t)1 << 31)
    return unsupported("max_pages * page_size must be in [1, 2^31)");
  if (b->max_new < 1 || b->max_kv < 0) return invalid("max_new must be positive, max_kv not negative");
  if (!stride_ok(b->table_stride, 1) || b->table_stride < b->max_pages)
    return invalid("table_stride must be at least max_pages");
  if (!b->q_start_dev || !b->kv_lens_dev || !b->page_table_dev) return invalid("null batch pointer");
  if (!aligned(b->q_start_dev, 4) || !aligned(b->kv_lens_dev, 4) || !aligned(b->page_table_dev, 4))
    return invalid("misaligned batch pointer");
  return OCQ_OK;
}

BatchArgs batch_args(const ocq_token_batch* b) {
  return BatchArgs{(const int32_t*)b->q_start_dev, (const int32_t*)b->kv_lens_dev, (const int32_t*)b->page_table_dev,
                   b->table_stride, b->requests, b->tokens, b->max_pages};
}

CacheArgs cache_args(const ocq_kv_cache* c) {
  const int64_t esz = c->format == OCQ_CACHE_E4M3 ? 1 : 2;
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  return CacheArgs{(uint8_t*)c->k_dev, (uint8_t*)c->v_dev, (float*)c->k_scale_dev, (float*)c->v_scale_dev,
                   c->head_stride * esz, c->scale_head_stride, (uint32_t)(c->page_stride * esz),
                   (uint32_t)(c->token_stride * esz), (uint32_t)c->scale_page_stride, (uint32_t)c->scale_token_stride,
                   c->num_pages, shift, c->kv_heads};
}

int max_new(const ocq_token_batch* b) { return b->max_new < b->tokens ? b->max_new : b->tokens; }

AttnPlan plan_of(int heads, const ocq_kv_cache* c, const ocq_token_batch* b, int window, int sinks) {
  return attn_plan(b->tokens, b->requests, max_new(b), b->max_kv, heads, c->kv_heads, c->head_dim, c->format, window,
                   sinks, (int64_t)b->max_pages * c->page_size);
}

}  // namespace

extern "C" {

ocq_status ocq_add_rmsnorm(const void* x_bf16_dev, int64_t x_stride, const void* residual_bf16_dev,
                           int64_t residual_stride, const void* weight_bf16_dev, float eps, int rows, int hidden,
                           void* residual_out_bf16_dev, void* y_bf16_dev, void* codes_dev, void* scales_dev,
                           void* stream) {
  set_error(OCQ_OK, "");
  if (rows < 0 || rows > (1 << 24)) return invalid("rows must be in [0, 2^24]");
  if (hidden < 8 || hidden > 65536 || hidden % 8) return unsupported("hidden must be a multiple of 8 in [8, 65536]");
  if (!(eps >= 0.0f) || std::isinf(eps)) return invalid("eps must be finite and not negative");
  if ((codes_dev == nullptr) != (scales_dev == nullptr)) return invalid("codes and scales go together");
  if (!y_bf16_dev && !codes_dev) return invalid("no output: y or codes and scales must be given");
  if (rows == 0) return OCQ_OK;
  if (!x_bf16_dev || !weight_bf16_dev) return invalid("null device pointer");
  const void* ptrs[] = {x_bf16_dev, residual_bf16_dev, weight_bf16_dev, residual_out_bf16_dev, y_bf16_dev, codes_dev};
  for (const void* p : ptrs)
    if (!aligned(p)) return invalid("device pointers must be 16-byte aligned");
  if (!aligned(scales_dev, 4)) return invalid("misaligned scale pointer");
  if (!stride_ok(x_stride, 8) || (residual_bf16_dev && !stride_ok(residual_stride, 8)))
    return invalid("row strides must be multiples of 8, not negative");
  const NormArgs a{(const uint16_t*)x_bf16_dev, (const uint16_t*)residual_bf16_dev, (const uint16_t*)weight_bf16_dev,
                   (uint16_t*)residual_out_bf16_dev, (uint16_t*)y_bf16_dev, (uint8_t*)codes_dev, (float*)scales_dev,
                   x_stride, residual_stride, eps, rows, hidden};
  const int rc = launch_norm(a, stream);
  return rc ? hip_error(rc) : OCQ_OK;
}

ocq_status ocq_rope_frequencies(int rot, double base, int scaling, double factor, double context, double beta_fast,
                                double beta_slow, double* inv_freq_out, float* multiplier_out) {
  set_error(OCQ_OK, "");
  if (rot < 16 || rot > 256 || rot % 16) return unsupported("rot must be a multiple of 16 in [16, 256]");
  if (scaling < OCQ_ROPE_PLAIN || scaling > OCQ_ROPE_YARN) return invalid("scaling must be 0, 1, 2 or 3");
  if (!(base > 1.0) || std::isinf(base) || !(factor >= 1.0) || std::isinf(factor))
    return invalid("base must be above 1 and factor at least 1, both finite");
  if (scaling == OCQ_ROPE_YARN &&
      (!(context > 0.0) || std::isinf(context) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || std::isinf(beta_fast)))
    return invalid("YaRN needs context > 0 and beta_fast > beta_slow > 0");
  if (!inv_freq_out || !multiplier_out) return invalid("null output pointer");
  if (scaling == OCQ_ROPE_NTK) base *= std::pow(factor, rot / (rot - 2.0));
  double low = 0.0, high = 0.0;
  if (scaling == OCQ_ROPE_YARN) {
    // j of the frequency that turns `t` times in `context` tokens
    const double two_pi = 6.283185307179586476925;
    auto turns = [&](double t) { return rot * std::log(context / (t * two_pi)) / (2.0 * std::log(base)); };
    low = std::fmax(0.0, std::floor(turns(beta_fast)));
    high = std::fmin(rot - 1.0, std::ceil(turns(beta_slow)));
  }
  for (int j = 0; j < rot / 2; ++j) {
    const double f = std::pow(base, -2.0 * j / rot);
    double keep = scaling == OCQ_ROPE_LINEAR ? 0.0 : 1.0;
    if (scaling == OCQ_ROPE_YARN) keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (j - low) / std::fmax(1e-3, high - low)));
    inv_freq_out[j] = f * keep + f / factor * (1.0 - keep);
  }
  *multiplier_out = scaling == OCQ_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return OCQ_OK;
}

ocq_status ocq_rope_append(const void* q_dev, int64_t q_token_stride, int64_t q_head_stride, const void* k_dev,
                           int64_t k_token_stride, int64_t k_head_stride, const void* v_dev, int64_t v_token_stride,
                           int64_t v_head_stride, int heads, const void* inv_freq_dev, int rot, int interleaved,
                           float multiplier, const void* positions_dev, const ocq_kv_cache* cache,
                           const ocq_token_batch* batch, void* q_out_dev, void* stream) {
  set_error(OCQ_OK, "");
  ocq_status st = check_cache(cache);
  if (st != OCQ_OK) return st;
  st = check_batch(batch, cache, heads);
  if (st != OCQ_OK) return st;
  if (rot < 16 || rot > cache->head_dim || rot % 16)
    return unsupported("rot must be a multiple of 16 in [16, head_dim]");
  if (interleaved != 0 && interleaved != 1) return invalid("interleaved must be 0 or 1");
  if (!std::isfinite(multiplier)) return invalid("multiplier must be finite");
  if (batch->requests == 0 || batch->tokens == 0) return OCQ_OK;
  if (!q_dev || !k_dev || !v_dev || !inv_freq_dev || !q_out_dev) return invalid("null device pointer");
  if (!aligned(q_dev) || !aligned(k_dev) || !aligned(v_dev) || !aligned(q_out_dev) || !aligned(inv_freq_dev, 8) ||
      !aligned(positions_dev, 4))
    return invalid("device pointers must be 16-byte aligned");
  const int64_t strides[] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  for (int64_t s : strides)
    if (!stride_ok(s, 8)) return invalid("strides must be multiples of 8, not negative");
  const RopeArgs a{(const uint16_t*)q_dev, (const uint16_t*)k_dev, (const uint16_t*)v_dev, q_token_stride,
                   q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                   (const double*)inv_freq_dev, (const int32_t*)positions_dev, (uint16_t*)q_out_dev, multiplier, heads,
                   cache->head_dim, rot, interleaved, cache->format == OCQ_CACHE_E4M3, 0, batch_args(batch),
                   cache_args(cache)};
  const int rc = launch_rope(a, stream);
  return rc ? hip_error(rc) : OCQ_OK;
}

size_t ocq_attention_workspace_bytes(int heads, const ocq_kv_cache* cache, const ocq_token_batch* batch, int window,
                                     int sinks) {
  set_error(OCQ_OK, "");
  if (check_cache(cache) != OCQ_OK || check_batch(batch, cache, heads) != OCQ_OK || window < 0 || sinks < 0) return 0;
  if (batch->requests == 0 || batch->tokens == 0) return 0;
  return plan_of(heads, cache, batch, window, sinks).part_rows * (cache->head_dim + 1) * sizeof(float);
}

ocq_status ocq_paged_attention(const void* q_dev, int64_t q_token_stride, int64_t q_head_stride, int heads,
                               const ocq_kv_cache* cache, const ocq_token_batch* batch, float scale, int window,
                               int sinks, void* out_dev, void* lse_dev, void* workspace_dev, size_t workspace_bytes,
                               void* stream) {
  set_error(OCQ_OK, "");
  ocq_status st = check_cache(cache);
  if (st != OCQ_OK) return st;
  st = check_batch(batch, cache, heads);
  if (st != OCQ_OK) return st;
  if (!(scale > 0.0f) || std::isinf(scale)) return invalid("scale must be positive and finite");
  if (window < 0 || sinks < 0 || (sinks > 0 && window == 0))
    return invalid("window and sinks must not be negative, and sinks need a window");
  if (batch->requests == 0 || batch->tokens == 0) return OCQ_OK;
  if (!q_dev || !out_dev || !batch->counters_dev) return invalid("null device pointer");
  if (!aligned(q_dev) || !aligned(out_dev) || !aligned(lse_dev, 4) || !aligned(batch->counters_dev, 4) || !aligned(workspace_dev))
    return invalid("device pointers must be 16-byte aligned");
  if (!stride_ok(q_token_stride, 8) || !stride_ok(q_head_stride, 8))
    return invalid("strides must be multiples of 8, not negative");
  const AttnPlan plan = plan_of(heads, cache, batch, window, sinks);
  if (plan.lanes >= 4294967296.0) return unsupported("too many row tiles for one launch");
  const size_t need = plan.part_rows * (cache->head_dim + 1) * sizeof(float);
  if (workspace_bytes < need)
    return set_error(OCQ_ERR_BUFFER_TOO_SMALL, "workspace_bytes < ocq_attention_workspace_bytes()");
  if (need && !workspace_dev) return invalid("null workspace");
  AttnArgs a{};
  a.q = (const uint16_t*)q_dev;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.out = (uint16_t*)out_dev;
  a.lse = (float*)lse_dev;
  a.scale = scale;
  a.heads = heads;
  a.group = heads / cache->kv_heads;
  a.dim = cache->head_dim;
  a.window = window;
  a.sinks = sinks;
  a.e4m3 = cache->format == OCQ_CACHE_E4M3;
  a.max_new = max_new(batch);
  a.b = batch_args(batch);
  a.c = cache_args(cache);
  a.even = plan.even;
  a.splits = plan.splits;
  a.groups = plan.groups;
  a.slots = plan.slots;
  a.counters = (uint32_t*)batch->counters_dev;
  a.part_o = (float*)workspace_dev;
  a.part_lse = (float*)workspace_dev + plan.part_rows * cache->head_dim;
  const int rc = launch_attn(a, stream);
  return rc ? hip_error(rc) : OCQ_OK;
}

}  // extern "C"
