// Calls of the C ABI between two verify steps that it must refuse, or that have
// nothing to do, under sanitizers: the launches are stand-ins that end the program
// if they are reached.
#include <cstdio>
#include <cstdlib>

#include "layer.h"
#include "ocq_internal.h"
#include "step.h"

namespace ocq {
ocq_status set_error(ocq_status st, const char*) { return st; }
[[noreturn]] static void unreachable() { std::abort(); }
int launch_values(const ValuesArgs&, void*) { unreachable(); }
int launch_drafts(const DraftArgs&, void*) { unreachable(); }
int launch_tables(const TableArgs&, void*) { unreachable(); }
DraftPlan draft_plan(int tokens, int requests, int, int) { return DraftPlan{1, 1, 0, 0, 0, (size_t)tokens * 64 + requests * 96}; }
size_t table_workspace(int requests, int tokens, int) { return tokens > 100 ? (size_t)requests * 32 : 0; }
}  // namespace ocq

static int failed = 0;
#define CHECK(x) do { if (!(x)) { ++failed; std::printf("line %d: %s\n", __LINE__, #x); } } while (0)

int main() {
  void* p = (void*)(uintptr_t)4096;   // never read
  ocq_kv_cache c{p, p, p, p, 8 * 16 * 64, 16 * 64, 64, 8 * 16 * 8, 16 * 8, 8, 7, 16, 8, 128, OCQ_CACHE_NVFP4, 0.5f, 4.0f};
  CHECK(ocq_cache_values(&c, p, nullptr, nullptr) == OCQ_ERR_INVALID_ARG);
  const float units[] = {0.0f, -1.0f, 3.0f, 1e-30f, 1e30f};
  for (float u : units) {
    c.v_unit = u;
    CHECK(ocq_cache_values(&c, p, p, nullptr) == OCQ_ERR_INVALID_ARG);
  }
  CHECK(ocq_cache_values(nullptr, p, p, nullptr) == OCQ_ERR_INVALID_ARG);

  const ocq_token_batch good{p, p, p, 9, 2, 5, 9, 3, 40, p};
  auto drafts = [&](const ocq_token_batch& b, int vocab, int64_t stride, float temp, size_t ws) {
    return ocq_verify_drafts(p, stride, 1, 0, p, stride, 3, 0, p, p, p, nullptr, temp, vocab, &b, p, p, p, ws, nullptr);
  };
  CHECK(ocq_verify_drafts_workspace_bytes(&good, 100, 0) == 5 * 64 + 2 * 96);
  CHECK(drafts(good, 100, 100, 1.0f, 511) == OCQ_ERR_BUFFER_TOO_SMALL);
  CHECK(drafts(good, 100, 99, 1.0f, 1 << 20) == OCQ_ERR_INVALID_ARG);
  CHECK(drafts(good, 0, 100, 1.0f, 1 << 20) == OCQ_ERR_UNSUPPORTED);
  CHECK(drafts(good, 100, 100, -1.0f, 1 << 20) == OCQ_ERR_INVALID_ARG);
  ocq_token_batch b = good;
  b.requests = OCQ_ATTENTION_COUNTERS + 1;
  CHECK(drafts(b, 100, 100, 1.0f, 1 << 20) == OCQ_ERR_UNSUPPORTED);
  b.requests = 0;
  CHECK(drafts(b, 100, 100, 1.0f, 0) == OCQ_OK);
  CHECK(ocq_verify_drafts_workspace_bytes(nullptr, 100, 0) == 0);

  const ocq_page_tables t{p, p, p, p, p, p, 8, 3, 8, 24, 16};
  auto step = [&](const ocq_page_tables& x, const ocq_page_tables& y, int tokens, size_t ws) {
    return ocq_step_tables(&x, &y, p, nullptr, tokens, p, p, p, p, p, ws, nullptr);
  };
  CHECK(ocq_step_tables_workspace_bytes(&t, 101) == 96 && ocq_step_tables_workspace_bytes(nullptr, 5) == 0);
  CHECK(step(t, t, 101, 95) == OCQ_ERR_BUFFER_TOO_SMALL);
  CHECK(step(t, t, -1, 0) == OCQ_ERR_INVALID_ARG);
  ocq_page_tables u = t;
  u.ring_size = 23;
  CHECK(step(t, u, 5, 0) == OCQ_ERR_INVALID_ARG);
  u = t;
  u.max_pages = 1 << 28;
  u.table_stride = 1 << 28;
  CHECK(step(u, u, 5, 0) == OCQ_ERR_UNSUPPORTED);
  u = t;
  u.requests = 0;
  CHECK(step(u, u, 5, 0) == OCQ_OK);
  std::printf("OK (%d failed checks)\n", failed);
  return failed != 0;
}
