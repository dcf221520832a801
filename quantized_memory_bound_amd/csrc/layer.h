// Internal declarations of the operators around the MLP block: residual +
// RMSNorm with an E4M3 output (norm.hip), rotary positions with the append to
// a paged cache (rope.hip), attention over that cache (attention.hip).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/ocq.h"

namespace ocq {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;       // nullable
  const uint16_t* w;
  uint16_t* res_out;         // nullable
  uint16_t* y;               // nullable
  uint8_t* codes;            // nullable
  float* scales;             // with codes
  int64_t x_stride, res_stride;   // elements between rows
  float eps;
  int rows, hidden;
};

// A token batch and a cache as the kernels take them (sizes checked by the
// entry points; contents of device arrays are bounded by the kernels).
struct BatchArgs {
  const int32_t* q_start;    // [requests + 1]
  const int32_t* kv_lens;    // [requests]
  const int32_t* table;      // [requests][table_stride]
  int64_t table_stride;
  int requests, tokens, max_pages;
};

struct CacheArgs {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;            // E4M3: one a row; NVFP4: E4M3 bytes, one per 16 values of a row
  float* v_scale;
  int64_t head, s_head;            // strides: of k and v in bytes, of the scales in elements (NVFP4: bytes)
  uint32_t page, token, s_page, s_token;
  int num_pages, page_shift, kv_heads;
  float k_unit, v_unit;      // NVFP4: what every scale is a multiple of
};

struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;   // strides in elements
  const double* inv_freq;    // [rot / 2]
  const int32_t* positions;  // nullable: place in the request
  uint16_t* q_out;           // [tokens][heads][dim]
  float multiplier;
  int heads, dim, rot, interleaved, format;
  int first;                 // token of the launch's first workgroup
  BatchArgs b;
  CacheArgs c;
};

struct AttnArgs {
  const uint16_t* q;
  int64_t q_token, q_head;   // strides in elements
  uint16_t* out;             // [tokens][heads][dim]
  float* lse;                // nullable, [tokens][heads]
  float scale;
  int heads, group, dim, window, sinks, format;
  int max_new;
  BatchArgs b;
  CacheArgs c;
  // work over the keys cut into pieces for `slots` workgroups (`groups` launched) or split `splits` ways;
  // partial outputs and their log2-sum-exps
  int even, splits, groups, slots;
  float* part_o;             // [part_rows][dim]
  float* part_lse;           // [part_rows]
  uint32_t* counters;        // [OCQ_ATTENTION_COUNTERS], 0 between calls
  // NVFP4 calls of many rows: room for every request's keys and values in fp16, `wide_pages`
  // pages a request, and for their page table; null: the codes are attended
  uint8_t* wide;
  int32_t* wide_table;
  int wide_pages;
  int wide_keys;             // keys of a request that these pages hold, max_kv at most
};

// The values that an E4M3 or NVFP4 cache stands for, [pages][kv_heads][page_size][dim] bf16.
struct ValuesArgs {
  uint16_t* k;
  uint16_t* v;
  int64_t rows;              // pages x kv_heads x page_size
  int dim, format;
  CacheArgs c;
};

struct AttnPlan {
  int even, splits, groups, slots;
  size_t part_rows;          // rows of partial outputs in the workspace
  double lanes = 0;          // of the larger launch (a launch holds fewer than 2^32)
};

// Pages a request whose keys and values a call over an NVFP4 cache widens to fp16
// first (0: it does not), and the bytes that they take.  Codes that every 32 rows
// convert for themselves keep the vector unit busy; widened once they cost a pass
// through memory.  32 heads of 128 on 8 kv heads, two requests over up to 10007 keys,
// us with and without: 512 rows a kv head 82 (67), 1024 113 (113), 2048 181 (187),
// 8192 469-498 (573); 16 requests, 2048 rows over 700 keys 117 (113).
constexpr int kWidened = 3;               // format of such a call's second launch
constexpr int kWideRows = 1024;
constexpr int64_t kWideBytes = (int64_t)1 << 30;
inline int64_t wide_bytes(int requests, int pages, int page_size, int kv_heads, int dim) {
  return (int64_t)requests * pages * ((int64_t)page_size * kv_heads * dim * 4 + 4);
}
inline int wide_pages(int format, int requests, int64_t rows, int max_kv, int max_pages, int page_size, int kv_heads,
                      int dim) {
  if (format != OCQ_CACHE_NVFP4 || rows < kWideRows) return 0;
  int64_t pages = ((int64_t)max_kv + page_size - 1) / page_size;
  pages = pages < max_pages ? pages : max_pages;
  // (a page of the widened cache is below 2^32 bytes, as of any cache)
  if (pages < 1 || (int64_t)page_size * kv_heads * dim * 2 > 0xFFFFFFFFll || (int64_t)requests * pages >= (int64_t)1 << 31 ||
      wide_bytes(requests, (int)pages, page_size, kv_heads, dim) > kWideBytes)
    return 0;
  return (int)pages;
}

// Lanes of one launch of the norm and the append (it holds fewer than 2^32); rows
// or tokens that take more are several launches.
constexpr unsigned kLanesAtOnce = 1u << 31;

// each enqueues on `stream` and returns 0 or a hipError_t value
int launch_norm(const NormArgs& a, void* stream);
int launch_rope(const RopeArgs& a, void* stream);
int launch_attn(const AttnArgs& a, void* stream);
int launch_values(const ValuesArgs& a, void* stream);
// layout of a call of this shape (host numbers only; cap: keys that a request's row of the page table can name)
AttnPlan attn_plan(int tokens, int requests, int max_new, int max_kv, int heads, int kv_heads, int dim, int format,
                   int window, int sinks, int64_t cap);

}  // namespace ocq
