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
  float* k_scale;            // E4M3 only
  float* v_scale;
  int64_t head, s_head;            // strides: of k and v in bytes, of the scales in elements
  uint32_t page, token, s_page, s_token;
  int num_pages, page_shift, kv_heads;
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
  int heads, dim, rot, interleaved, e4m3;
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
  int heads, group, dim, window, sinks, e4m3;
  int max_new;
  BatchArgs b;
  CacheArgs c;
  // work over the keys cut into pieces for `slots` workgroups (`groups` launched) or split `splits` ways;
  // partial outputs and their log2-sum-exps
  int even, splits, groups, slots;
  float* part_o;             // [part_rows][dim]
  float* part_lse;           // [part_rows]
  uint32_t* counters;        // [OCQ_ATTENTION_COUNTERS], 0 between calls
};

struct AttnPlan {
  int even, splits, groups, slots;
  size_t part_rows;          // rows of partial outputs in the workspace
  double lanes = 0;          // of the larger launch (a launch holds fewer than 2^32)
};

// Lanes of one launch of the norm and the append (it holds fewer than 2^32); rows
// or tokens that take more are several launches.
constexpr unsigned kLanesAtOnce = 1u << 31;

// each enqueues on `stream` and returns 0 or a hipError_t value
int launch_norm(const NormArgs& a, void* stream);
int launch_rope(const RopeArgs& a, void* stream);
int launch_attn(const AttnArgs& a, void* stream);
// layout of a call of this shape (host numbers only; cap: keys that a request's row of the page table can name)
AttnPlan attn_plan(int tokens, int requests, int max_new, int max_kv, int heads, int kv_heads, int dim, int e4m3,
                   int window, int sinks, int64_t cap);

}  // namespace ocq
