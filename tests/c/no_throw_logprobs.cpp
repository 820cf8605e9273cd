// The log-probability and clipping entry points with allocations that fail, from the first,
// the second and so on of each call: no exception may leave a C function.  Calls that need
// no GPU: size queries, refusals, and calls that DMUON_TEST_FAIL_AT=plan ends before a launch.
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
  const auto f = [&](int i) { return (float*)at(i); };
  dmuon_logprobs_problem p = {3, 50000, DMUON_BF16, DMUON_I64, at(1), 50000, at(2), -100, 1.f, 5};
  dmuon_logprobs_problem bad = p;
  bad.scale = 0.f;
  dmuon_ce_problem ce = {64, 128, 1000, DMUON_BF16, DMUON_I64, at(1), 128, at(2), 128, at(3), -100};
  dmuon_grad_tensor t[2] = {{1000, DMUON_BF16, DMUON_F32, at(1), at(2)}, {70000, DMUON_F32, DMUON_F32, at(3), at(3)}};
  dmuon_grad_tensor bad_t[1] = {{-1, DMUON_BF16, DMUON_F32, at(1), at(2)}};
  void* ws = at(20);
  const size_t big = (size_t)1 << 38;
  size_t bytes = 0;
  each("rows size", [&] { return dmuon_logprobs_workspace_size(&p, &bytes); });
  each("rows size refused", [&] { return dmuon_logprobs_workspace_size(&bad, &bytes); });
  each("rows", [&] { return dmuon_logprobs(&p, f(3), f(4), f(5), (int64_t*)at(6), f(7), ws, big, nullptr); });
  each("rows refused", [&] { return dmuon_logprobs(&p, f(3), f(3), f(5), (int64_t*)at(6), f(7), ws, big, nullptr); });
  each("rows backward", [&] { return dmuon_logprobs_backward(&p, f(5), f(4), f(8), f(9), at(10), 50000, nullptr); });
  each("rows backward refused", [&] { return dmuon_logprobs_backward(&p, f(5), f(4), f(8), f(9), at(2), 50000, nullptr); });
  each("linear size", [&] { return dmuon_linear_logprobs_workspace_size(&ce, 1, &bytes); });
  each("linear", [&] { return dmuon_linear_logprobs(&ce, 1.f, f(4), f(5), f(6), ws, big, nullptr); });
  each("linear refused", [&] { return dmuon_linear_logprobs(&ce, 0.f, f(4), f(5), f(6), ws, big, nullptr); });
  each("linear backward", [&] { return dmuon_linear_logprobs_backward(&ce, 1.f, f(6), f(5), f(7), f(8), at(9), at(10), ws, big, nullptr); });
  each("clip size", [&] { return dmuon_grad_workspace_size(t, 2, &bytes); });
  each("clip size refused", [&] { return dmuon_grad_workspace_size(bad_t, 1, &bytes); });
  each("clip prepare", [&] { return dmuon_grad_prepare(t, 2, ws, big, nullptr); });
  each("norm", [&] { return dmuon_grad_norm_run(t, 2, f(9), ws, big, nullptr); });
  each("clip", [&] { return dmuon_grad_clip_run(t, 2, 1.f, 0.f, 1, f(9), ws, big, nullptr); });
  each("clip refused", [&] { return dmuon_grad_clip_run(t, 2, 1.f, 0.f, 1, f(2), ws, big, nullptr); });
  std::puts("ok");
}
