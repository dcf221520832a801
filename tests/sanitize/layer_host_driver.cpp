// Calls of the layer operators' C ABI that it must refuse, under sanitizers:
// the launches are stand-ins that end the program if they are reached.
#include <cstdio>
#include <cstdlib>

#include "layer.h"
#include "ocq_internal.h"

namespace ocq {
ocq_status set_error(ocq_status st, const char*) { return st; }
[[noreturn]] static void unreachable() { std::abort(); }
int launch_norm(const NormArgs&, void*) { unreachable(); }
int launch_rope(const RopeArgs&, void*) { unreachable(); }
int launch_attn(const AttnArgs&, void*) { unreachable(); }
AttnPlan attn_plan(int tokens, int, int, int, int heads, int, int, int, int, int, int64_t) {
  return AttnPlan{0, 3, 0, 0, (size_t)3 * tokens * heads};
}
}  // namespace ocq

static int failed = 0;
#define CHECK(x) do { if (!(x)) { ++failed; std::printf("line %d: %s\n", __LINE__, #x); } } while (0)

int main() {
  void* p = (void*)(uintptr_t)4096;   // never read: every call is refused or has nothing to do
  double inv[128];
  float mult = 0.0f;
  for (int rot = 16; rot <= 256; rot += 16)
    for (int kind = 0; kind < 4; ++kind) {
      CHECK(ocq_rope_frequencies(rot, 1e4, kind, 8.0, 4096.0, 32.0, 1.0, inv, &mult) == OCQ_OK);
      for (int j = 0; j < rot / 2; ++j) CHECK(inv[j] > 0.0 && inv[j] <= 1.0);
    }
  CHECK(ocq_rope_frequencies(24, 1e4, 0, 1, 1, 2, 1, inv, &mult) == OCQ_ERR_UNSUPPORTED);
  const ocq_kv_cache good{p, p, p, p, 8 * 16 * 128, 16 * 128, 128, 128, 16, 1, 7, 16, 8, 128, OCQ_CACHE_E4M3};
  const ocq_token_batch step{p, p, p, 9, 2, 5, 9, 3, 40, p};
  auto attn = [&](const ocq_kv_cache& c, const ocq_token_batch& b, int heads, float scale, int window, int sinks,
                  size_t ws) {
    return ocq_paged_attention(p, 4096, 128, heads, &c, &b, scale, window, sinks, p, p, p, ws, nullptr);
  };
  CHECK(attn(good, step, 32, 0.1f, 0, 0, 0) == OCQ_ERR_BUFFER_TOO_SMALL);
  CHECK(ocq_attention_workspace_bytes(32, &good, &step, 0, 0) == (size_t)3 * 5 * 32 * 129 * 4);
  CHECK(attn(good, step, 32, 0.0f, 0, 0, 1 << 30) == OCQ_ERR_INVALID_ARG);
  CHECK(attn(good, step, 32, 0.1f, 0, 4, 1 << 30) == OCQ_ERR_INVALID_ARG);
  CHECK(attn(good, step, 33, 0.1f, 0, 0, 1 << 30) == OCQ_ERR_INVALID_ARG);
  ocq_kv_cache c = good;
  c.page_size = 24;
  CHECK(attn(c, step, 32, 0.1f, 0, 0, 1 << 30) == OCQ_ERR_UNSUPPORTED);
  c = good;
  c.token_stride = 136;   // 136 bytes of codes: not 16-byte aligned rows
  CHECK(attn(c, step, 32, 0.1f, 0, 0, 1 << 30) == OCQ_ERR_INVALID_ARG);
  ocq_token_batch b = step;
  b.max_pages = 1 << 28;
  CHECK(attn(good, b, 32, 0.1f, 0, 0, 1 << 30) == OCQ_ERR_UNSUPPORTED);
  b = step;
  b.tokens = 0;
  CHECK(attn(good, b, 32, 0.1f, 0, 0, 0) == OCQ_OK);   // nothing to do
  CHECK(ocq_add_rmsnorm(p, 64, nullptr, 0, p, 1e-6f, 0, 64, nullptr, p, nullptr, nullptr, nullptr) == OCQ_OK);
  CHECK(ocq_add_rmsnorm(p, 64, nullptr, 0, p, 1e-6f, 1, 60, nullptr, p, nullptr, nullptr, nullptr) ==
        OCQ_ERR_UNSUPPORTED);
  std::printf("OK (%d failed checks)\n", failed);
  return failed != 0;
}
