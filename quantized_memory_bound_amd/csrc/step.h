// Internal declarations of what stands between two verify steps: which drafts
// stay and the token after them (drafts.hip), the next step's tables (tables.hip).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/ocq.h"

namespace ocq {

struct RowStat;   // drafts.hip
struct RowDraft;
struct Choice;

struct DraftArgs {
  const void* target;        // [tokens][vocab]: logits or probabilities
  const void* draft;         // nullable, [draft_rows][vocab]: the draft's probabilities
  int64_t t_stride, d_stride, draft_rows;
  const int32_t* ids;        // [tokens]
  const float* u_accept;     // [tokens]
  const float* u_next;       // [requests]
  const float* temps;        // nullable, [requests]
  float temp;
  const int32_t* q_start;
  int requests, tokens, vocab;
  int t_bf16, d_bf16, probs;
  int32_t* accepted;         // [requests]
  int32_t* out;              // [tokens]
  int splits, chunks;        // workgroups of a row's statistics, and of a request's drawn row
  RowStat* stats;            // [tokens][splits]
  RowDraft* row_drafts;      // [tokens]
  Choice* choices;           // [requests]
  double* parts;             // [requests][chunks][4]: sums of the drawn row
  uint32_t* counters;        // [OCQ_ATTENTION_COUNTERS], 0 between calls
};

struct DraftPlan {
  int splits, chunks;
  size_t drafts_at, choices_at, parts_at, bytes;   // of the workspace
};
DraftPlan draft_plan(int tokens, int requests, int vocab, int probs);

struct TableArgs {
  const int32_t* q_in;       // [requests + 1], of the step before
  const int32_t* kv_in;
  const int32_t* held_in;
  const int64_t* counts_in;  // ring entries taken, given
  const int32_t* news;
  const int32_t* accepted;   // nullable: all tokens of the step before stay
  int32_t* q_out;            // may be the inputs
  int32_t* kv_out;
  int32_t* held_out;
  int64_t* counts_out;
  int32_t* table;
  int32_t* ring;
  int64_t table_stride;
  int64_t* slots;            // [tokens], nullable like the next two
  int32_t* positions;
  int32_t* owners;
  int32_t* missing;          // [1]
  int requests, tokens, max_pages, ring_size, page_shift;
  int32_t* records;          // workspace of a step in two launches
};
size_t table_workspace(int requests, int tokens, int max_pages);

// each enqueues on `stream` and returns 0 or a hipError_t value
int launch_drafts(const DraftArgs& a, void* stream);
int launch_tables(const TableArgs& a, void* stream);

}  // namespace ocq
