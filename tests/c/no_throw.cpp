// Every training-gradient entry point with allocations that fail, from the first, the second
// and so on of its call: no exception may leave a C function.  Calls that need no GPU:
// size queries, refusals, and calls that DMUON_TEST_FAIL_AT=plan ends before a launch.
#include <cstdio>
#include <cstdlib>
#include <new>

#include "dmuon_ns.h"

static long left = -1;                        // allocations until they fail; < 0: none does
static bool failed = false;

void* operator new(std::size_t n) {
  if (left == 0) {
    failed = true;
    throw std::bad_alloc();
  }
  if (left > 0) --left;
  if (void* p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

template <typename F>
static void each(const char* what, F&& call) {
  int most = 0;
  for (long n = 0;; ++n) {
    left = n;
    failed = false;
    const int rc = call();
    left = -1;
    const char* text = dmuon_last_error();
    if (!failed) break;                       // the call has no more than n allocations
    most = (int)n + 1;
    if (rc != DMUON_E_HIP || !text || !*text) {
      std::printf("%s: allocation %ld failed, the call returned %d \"%s\"\n", what, n, rc, text ? text : "(null)");
      std::exit(1);
    }
    if (n > 200) std::exit(2);
  }
  std::printf("%s: %d allocations\n", what, most);
}

int main() {
  const auto at = [](int i) { return (char*)0x7f0000000000 + ((size_t)i << 40); };
  dmuon_ce_problem ce = {64, 128, 1000, DMUON_BF16, DMUON_I64, at(1), 128, at(2), 128, at(3), -100};
  dmuon_ce_problem bad = ce;
  bad.vocab = 0;
  dmuon_ckpt8_wgrad_problem wg = {64, 100, 200, DMUON_BF16, DMUON_F32, at(1), 100, (const int8_t*)at(2), (const uint8_t*)at(3),
                                  nullptr, 0, 0, at(4)};
  dmuon_ckpt8_wgrad_problem bad_wg = wg;
  bad_wg.reserved = 1;
  float *f4 = (float*)at(4), *f5 = (float*)at(5), *f6 = (float*)at(6);
  void* ws = at(20);
  const size_t big = (size_t)1 << 38;
  size_t bytes = 0;
  each("ce size", [&] { return dmuon_linear_ce_workspace_size(&ce, 1, &bytes); });
  each("ce size refused", [&] { return dmuon_linear_ce_workspace_size(&bad, 0, &bytes); });
  each("ce", [&] { return dmuon_linear_ce(&ce, f4, f5, ws, big, nullptr); });
  each("ce refused", [&] { return dmuon_linear_ce(&ce, f4, f4, ws, big, nullptr); });
  each("ce backward", [&] { return dmuon_linear_ce_backward(&ce, f5, f6, at(7), at(8), ws, big, nullptr); });
  each("ce backward refused", [&] { return dmuon_linear_ce_backward(&ce, f5, f6, at(1), at(8), ws, big, nullptr); });
  each("embedding", [&] { return dmuon_embedding(at(1), DMUON_I64, 10, at(2), 64, 100, 64, DMUON_BF16, 1.f, at(3), nullptr); });
  each("embedding refused", [&] { return dmuon_embedding(at(1), DMUON_I64, 10, at(2), 63, 100, 64, DMUON_BF16, 1.f, at(3), nullptr); });
  each("embedding backward size", [&] { return dmuon_embedding_backward_workspace_size(10, 100, 64, &bytes); });
  each("embedding backward", [&] {
    return dmuon_embedding_backward(at(1), DMUON_I64, 10, at(2), 64, DMUON_BF16, 100, 64, 1.f, -1, at(3), DMUON_F32, 0, ws, big, nullptr);
  });
  each("embedding backward refused", [&] {
    return dmuon_embedding_backward(at(1), DMUON_I64, 10, at(2), 64, DMUON_BF16, 100, 64, 1.f, -1, at(3), DMUON_F32, 0, ws, 1, nullptr);
  });
  each("quantize", [&] { return dmuon_ckpt8_quantize(at(1), DMUON_BF16, 4, 64, 64, (int8_t*)at(2), (uint8_t*)at(3), nullptr); });
  each("dequantize", [&] { return dmuon_ckpt8_dequantize((int8_t*)at(2), (uint8_t*)at(3), 4, 64, at(1), 7, nullptr); });
  each("wgrad size", [&] { return dmuon_ckpt8_wgrad_workspace_size(&wg, &bytes); });
  each("wgrad", [&] { return dmuon_ckpt8_wgrad(&wg, ws, big, nullptr); });
  each("wgrad refused", [&] { return dmuon_ckpt8_wgrad(&bad_wg, ws, big, nullptr); });
  std::puts("ok");
}
