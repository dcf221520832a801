// C-ABI entry points of what stands between two verify steps: the values of a
// quantized cache, the drafts that stay and the token after them, the next
// step's tables.
#include "layer_check.h"
#include "step.h"

using namespace ocq;

namespace {

ocq_status check_rows(const ocq_token_batch* b) {
  if (!b) return invalid("batch is null");
  if (b->requests < 0 || b->tokens < 0) return invalid("requests and tokens must not be negative");
  if (b->requests > OCQ_ATTENTION_COUNTERS) return unsupported("at most OCQ_ATTENTION_COUNTERS requests");
  if (b->tokens > 1 << 20) return unsupported("at most 2^20 tokens");
  if (b->requests == 0 || b->tokens == 0) return OCQ_OK;
  if (!b->q_start_dev || !b->counters_dev) return invalid("null batch pointer");
  if (!aligned(b->q_start_dev, 4) || !aligned(b->counters_dev, 4)) return invalid("misaligned batch pointer");
  return OCQ_OK;
}
ocq_status check_vocab(int vocab) {
  return vocab >= 1 && vocab <= 1 << 24 ? OCQ_OK : unsupported("vocab must be in [1, 2^24]");
}

ocq_status check_tables(const ocq_page_tables* t) {
  if (!t) return invalid("tables are null");
  if (t->requests < 0 || t->requests > 65536) return unsupported("requests must be in [0, 65536]");
  if (t->page_size < 1 || t->page_size > 1024 || (t->page_size & (t->page_size - 1)))
    return unsupported("page_size must be a power of two in [1, 1024]");
  if (t->max_pages < 1 || (int64_t)t->max_pages * t->page_size >= (int64_t)1 << 31)
    return unsupported("max_pages * page_size must be in [1, 2^31)");
  // (a lane's next page is up to 2^14 places on, in 32 bits; so are the sums over the
  // requests of the pages that they take and give: past that two would get one page)
  if (t->max_pages > 1 << 30) return unsupported("at most 2^30 pages a request");
  if ((int64_t)t->requests * t->max_pages >= (int64_t)1 << 31) return unsupported("requests * max_pages must be below 2^31");
  if (t->ring_size < 1) return invalid("ring_size must be positive");
  if (!stride_ok(t->table_stride, 1) || t->table_stride < t->max_pages)
    return invalid("table_stride must be at least max_pages");
  const void* ptrs[] = {t->q_start_dev, t->kv_lens_dev, t->held_dev, t->page_table_dev, t->ring_dev};
  for (const void* p : ptrs) {
    if (!p) return invalid("null table pointer");
    if (!aligned(p, 4)) return invalid("misaligned table pointer");
  }
  if (!t->counts_dev || !aligned(t->counts_dev, 8)) return invalid("counts must be an 8-byte aligned pointer");
  return OCQ_OK;
}

}  // namespace

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

size_t ocq_verify_drafts_workspace_bytes(const ocq_token_batch* batch, int vocab, int probabilities) {
  set_error(OCQ_OK, "");
  if (check_rows(batch) != OCQ_OK || check_vocab(vocab) != OCQ_OK) return 0;
  if (batch->requests == 0 || batch->tokens == 0) return 0;
  return draft_plan(batch->tokens, batch->requests, vocab, probabilities != 0).bytes;
}

ocq_status ocq_verify_drafts(const void* target_dev, int64_t target_stride, int target_bf16, int probabilities,
                             const void* draft_dev, int64_t draft_stride, int64_t draft_rows, int draft_bf16,
                             const void* tokens_dev, const void* u_accept_dev, const void* u_next_dev,
                             const void* temperature_dev, float temperature, int vocab, const ocq_token_batch* batch,
                             void* accepted_dev, void* out_dev, void* workspace_dev, size_t workspace_bytes,
                             void* stream) {
  set_error(OCQ_OK, "");
  ocq_status st = check_rows(batch);
  if (st != OCQ_OK) return st;
  st = check_vocab(vocab);
  if (st != OCQ_OK) return st;
  if ((target_bf16 | draft_bf16 | probabilities) & ~1) return invalid("target_bf16, draft_bf16 and probabilities are 0 or 1");
  if (!probabilities && !temperature_dev && !(temperature >= 0.0f && std::isfinite(temperature)))
    return invalid("temperature must be finite and not negative");
  if (batch->requests == 0 || batch->tokens == 0) return OCQ_OK;
  if (!target_dev || !tokens_dev || !u_accept_dev || !u_next_dev || !accepted_dev || !out_dev)
    return invalid("null device pointer");
  const void* ptrs[] = {tokens_dev, u_accept_dev, u_next_dev, temperature_dev, accepted_dev, out_dev};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return invalid("misaligned device pointer");
  if (!aligned(target_dev, target_bf16 ? 2 : 4) || !aligned(draft_dev, draft_bf16 ? 2 : 4))
    return invalid("misaligned device pointer");
  if (!stride_ok(target_stride, 1) || (batch->tokens > 1 && target_stride < vocab) ||
      (draft_dev && (!stride_ok(draft_stride, 1) || (draft_rows > 1 && draft_stride < vocab) || draft_rows < 0)))
    return invalid("rows must lie vocab elements or more apart");
  const DraftPlan plan = draft_plan(batch->tokens, batch->requests, vocab, probabilities);
  if (workspace_bytes < plan.bytes)
    return set_error(OCQ_ERR_BUFFER_TOO_SMALL, "workspace_bytes < ocq_verify_drafts_workspace_bytes()");
  if (!workspace_dev || !aligned(workspace_dev)) return invalid("the workspace must be a 16-byte aligned pointer");
  DraftArgs a{};
  a.target = target_dev;
  a.draft = draft_dev;
  a.t_stride = target_stride;
  a.d_stride = draft_stride;
  a.draft_rows = draft_rows;
  a.ids = (const int32_t*)tokens_dev;
  a.u_accept = (const float*)u_accept_dev;
  a.u_next = (const float*)u_next_dev;
  a.temps = (const float*)temperature_dev;
  a.temp = temperature;
  a.q_start = (const int32_t*)batch->q_start_dev;
  a.requests = batch->requests;
  a.tokens = batch->tokens;
  a.vocab = vocab;
  a.t_bf16 = target_bf16;
  a.d_bf16 = draft_bf16;
  a.probs = probabilities;
  a.accepted = (int32_t*)accepted_dev;
  a.out = (int32_t*)out_dev;
  a.splits = plan.splits;
  a.chunks = plan.chunks;
  a.stats = (RowStat*)workspace_dev;
  a.row_drafts = (RowDraft*)((uint8_t*)workspace_dev + plan.drafts_at);
  a.choices = (Choice*)((uint8_t*)workspace_dev + plan.choices_at);
  a.parts = (double*)((uint8_t*)workspace_dev + plan.parts_at);
  a.counters = (uint32_t*)batch->counters_dev;
  const int rc = launch_drafts(a, stream);
  return rc ? hip_error(rc) : OCQ_OK;
}

size_t ocq_step_tables_workspace_bytes(const ocq_page_tables* tables, int tokens) {
  set_error(OCQ_OK, "");
  if (check_tables(tables) != OCQ_OK || tokens < 0 || tokens > 1 << 30) return 0;
  return table_workspace(tables->requests, tokens, tables->max_pages);
}

ocq_status ocq_step_tables(const ocq_page_tables* before, const ocq_page_tables* after, const void* news_dev,
                           const void* accepted_dev, int tokens, void* slots_dev, void* positions_dev,
                           void* requests_dev, void* missing_dev, void* workspace_dev, size_t workspace_bytes,
                           void* stream) {
  set_error(OCQ_OK, "");
  ocq_status st = check_tables(before);
  if (st != OCQ_OK) return st;
  st = check_tables(after);
  if (st != OCQ_OK) return st;
  if (before->page_table_dev != after->page_table_dev || before->ring_dev != after->ring_dev ||
      before->table_stride != after->table_stride || before->requests != after->requests ||
      before->max_pages != after->max_pages || before->ring_size != after->ring_size ||
      before->page_size != after->page_size)
    return invalid("before and after share one page table and one ring, and their sizes");
  if (tokens < 0) return invalid("tokens must not be negative");
  // (a lane's next token is up to 2^16 places on, in 32 bits)
  if (tokens > 1 << 30) return unsupported("at most 2^30 tokens");
  if (before->requests == 0) return OCQ_OK;
  if (!news_dev) return invalid("null device pointer");
  const void* ptrs[] = {news_dev, accepted_dev, positions_dev, requests_dev, missing_dev};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return invalid("misaligned device pointer");
  if (!aligned(slots_dev, 8)) return invalid("slots must be 8-byte aligned");
  const size_t need = table_workspace(before->requests, tokens, before->max_pages);
  if (workspace_bytes < need)
    return set_error(OCQ_ERR_BUFFER_TOO_SMALL, "workspace_bytes < ocq_step_tables_workspace_bytes()");
  if (need && (!workspace_dev || !aligned(workspace_dev))) return invalid("the workspace must be a 16-byte aligned pointer");
  TableArgs a{};
  a.q_in = (const int32_t*)before->q_start_dev;
  a.kv_in = (const int32_t*)before->kv_lens_dev;
  a.held_in = (const int32_t*)before->held_dev;
  a.counts_in = (const int64_t*)before->counts_dev;
  a.news = (const int32_t*)news_dev;
  a.accepted = (const int32_t*)accepted_dev;
  a.q_out = (int32_t*)after->q_start_dev;
  a.kv_out = (int32_t*)after->kv_lens_dev;
  a.held_out = (int32_t*)after->held_dev;
  a.counts_out = (int64_t*)after->counts_dev;
  a.table = (int32_t*)before->page_table_dev;
  a.ring = (int32_t*)before->ring_dev;
  a.table_stride = before->table_stride;
  a.slots = (int64_t*)slots_dev;
  a.positions = (int32_t*)positions_dev;
  a.owners = (int32_t*)requests_dev;
  a.missing = (int32_t*)missing_dev;
  a.requests = before->requests;
  a.tokens = tokens;
  a.max_pages = before->max_pages;
  a.ring_size = before->ring_size;
  while ((1 << a.page_shift) < before->page_size) ++a.page_shift;
  a.records = (int32_t*)workspace_dev;
  const int rc = launch_tables(a, stream);
  return rc ? hip_error(rc) : OCQ_OK;
}

}  // extern "C"
