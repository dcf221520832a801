// C-ABI entry points of what stands between two verify steps: the values of a
// quantized cache.
#include "layer_check.h"

using namespace ocq;

extern "C" {

ocq_status ocq_cache_values(const ocq_kv_cache* cache, void* k_out_dev, void* v_out_dev, void* stream) {
  set_error(OCQ_OK, "");
  const ocq_status st = check_cache(cache);
  if (st != OCQ_OK) return st;
  if (cache->format == OCQ_CACHE_BF16) return invalid("a bf16 cache holds its values");
  if (!k_out_dev || !v_out_dev) return invalid("null device pointer");
  if (!aligned(k_out_dev) || !aligned(v_out_dev)) return invalid("device pointers must be 16-byte aligned");
  const ValuesArgs a{(uint16_t*)k_out_dev, (uint16_t*)v_out_dev,
                     (int64_t)cache->num_pages * cache->kv_heads * cache->page_size, cache->head_dim, cache->format,
                     cache_args(cache)};
  const int rc = launch_values(a, stream);
  return rc ? hip_error(rc) : OCQ_OK;
}

}  // extern "C"
