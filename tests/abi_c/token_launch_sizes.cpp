// Grids of the launches of embedding, dropout and log probabilities at the
// largest sizes the C ABI accepts.  This program defines hipLaunchKernel itself, so
// nothing runs on a GPU: every launch is recorded and must hold fewer than 2^32 work
// items in each dimension, and a call's launches together as many workgroups as its
// rows need.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <vector>

#include "gc.h"

namespace {

struct Launch {
  dim3 grid, block;
};
std::vector<Launch> g_launches;
int g_failures = 0;

uint64_t g_at = uint64_t(1) << 44;
// A stand-in device address with room for 2^40 bytes behind it.
void* buf() { return reinterpret_cast<void*>(g_at += uint64_t(1) << 41); }
std::vector<void*> g_lists;
template <class T = void>
T* const* out() {
  g_lists.push_back(buf());
  return reinterpret_cast<T* const*>(&g_lists.back());
}
template <class T = void>
const T* const* in() { return const_cast<const T* const*>(out<T>()); }

// Ends a call: `least` workgroups in all, of whatever kernels.
void check(const char* what, gc_status s, uint64_t least, gc_status want = GC_OK) {
  uint64_t blocks = 0;
  bool fits = true;
  for (const Launch& l : g_launches) {
    blocks += uint64_t(l.grid.x) * l.grid.y;
    fits &= uint64_t(l.grid.x) * l.block.x < (uint64_t(1) << 32) && uint64_t(l.grid.y) * l.block.y < (uint64_t(1) << 32);
    fits &= l.grid.x > 0 && l.grid.y > 0;
  }
  const bool ok = s == want && fits && blocks >= least && (want == GC_OK || g_launches.empty());
  std::printf("%-46s status %d, %zu launches, %llu workgroups: %s\n", what, s, g_launches.size(),
              static_cast<unsigned long long>(blocks), ok ? "ok" : "FAILED");
  if (!ok) ++g_failures;
  g_launches.clear();
}

void lookup(const char* what, int64_t n, size_t vocab, size_t hidden, gc_dtype t, uint64_t least) {
  check(what, gc_embedding(in(), in<int32_t>(), &n, 1, vocab, hidden, 1.0f, t, out(), nullptr), least);
}

void gradient(const char* what, int64_t n, size_t vocab, size_t hidden, gc_dtype t, gc_dtype wt, uint64_t least) {
  const size_t need = gc_embedding_backward_scratch_bytes(&n, 1, vocab, hidden);
  check(what, gc_embedding_backward(in(), in<int32_t>(), &n, 1, vocab, hidden, 1.0f, t, out(), wt, 0, buf(), need, nullptr), least);
}

void rows(const char* what, int64_t n, size_t vocab, int top, gc_dtype t, uint64_t least) {
  const size_t need = gc_token_logprob_scratch_bytes(&n, 1, vocab, top);
  check(what, gc_token_logprob(in(), in<int32_t>(), &n, 1, vocab, vocab, 1.0f, t, out<float>(), nullptr, nullptr, top, out<int32_t>(),
                               out<float>(), nullptr, nullptr, nullptr, buf(), need, nullptr), least);
  check(what, gc_token_logprob_backward(in(), in<int32_t>(), in<float>(), nullptr, in<float>(), nullptr, &n, 1, vocab, vocab, 1.0f, t, out(),
                                        nullptr), least);
}

}  // namespace

extern "C" hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
  g_launches.push_back({grid, block});
  return hipSuccess;
}

int main() {
  g_lists.reserve(4096);
  const int64_t most = (int64_t(1) << 31) - 1;
  lookup("lookup, 2^31 - 1 rows of 1", most, 1, 1, GC_FP32, 1 << 23);
  lookup("lookup, 2^31 - 1 rows of 64", most, 1000, 64, GC_BF16, 1 << 26);
  lookup("lookup, 5 rows of 2^31", 5, 1, size_t(1) << 31, GC_BF16, 5 << 18);
  lookup("lookup, 2^26 + 3 rows of 4096", (int64_t(1) << 26) + 3, 5000, 4096, GC_BF16, 1 << 25);
  gradient("gradient, 2^31 - 1 rows of 1", most, 5, 1, GC_FP32, GC_FP32, 1 << 20);
  gradient("gradient, 2^22 x 70000 of 3 rows", 3, size_t(1) << 22, 70000, GC_BF16, GC_BF16, 1 << 22);
  gradient("gradient, 2^26 + 3 rows of 512", (int64_t(1) << 26) + 3, 1 << 16, 512, GC_BF16, GC_FP32, 1 << 18);
  gradient("gradient, 3 rows of 2^31", 3, 4, size_t(1) << 31, GC_FP32, GC_FP32, 1 << 19);
  for (int64_t n : {int64_t(1) << 32, (int64_t(1) << 38) + 9})
    check("dropout of 2^32 and 2^38 + 9 elements",
          gc_dropout(in(), nullptr, &n, 1, 0.1f, 1, 0, nullptr, GC_BF16, out(), nullptr), static_cast<uint64_t>(n) / 2048);
  rows("rows, 2^31 - 1 of 1", most, 1, 0, GC_BF16, 1 << 29);
  rows("rows, 2^31 - 1 of 100 with 5", most, 100, 5, GC_BF16, 1 << 29);
  rows("rows, 2^24 + 1 of 30000 with 64", (int64_t(1) << 24) + 1, 30000, 64, GC_BF16, (1 << 24) + 1);
  rows("rows, 2 of 2^31 with 3", 2, size_t(1) << 31, 3, GC_FP32, 2);
  std::printf("%d failures\n", g_failures);
  return g_failures != 0;
}
