// Grids of the library's launches at the largest sizes the C ABI accepts.  This
// program defines hipLaunchKernel itself, so nothing runs on a GPU: every launch
// is recorded and must hold fewer than 2^32 work items in each dimension, and a
// call's launches together as many workgroups as its rows need.
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
void* const* list() {
  g_lists.push_back(buf());
  return &g_lists.back();
}
template <class T>
const T* const* in() { return reinterpret_cast<const T* const*>(list()); }

// Ends a call: `least` workgroups in all, of whatever kernels.
void check(const char* what, gc_status s, uint64_t least) {
  uint64_t blocks = 0;
  bool fits = true;
  for (const Launch& l : g_launches) {
    blocks += uint64_t(l.grid.x) * l.grid.y;
    fits &= uint64_t(l.grid.x) * l.block.x < (uint64_t(1) << 32) && uint64_t(l.grid.y) * l.block.y < (uint64_t(1) << 32);
    fits &= l.grid.x > 0 && l.grid.y > 0;
  }
  const bool ok = s == GC_OK && fits && blocks >= least;
  std::printf("%-40s status %d, %zu launches, %llu workgroups: %s\n", what, s, g_launches.size(),
              static_cast<unsigned long long>(blocks), ok ? "ok" : "FAILED");
  if (!ok) ++g_failures;
  g_launches.clear();
}

void norm(const char* what, int64_t rows, size_t hidden, gc_dtype t, gc_dtype yt, uint64_t least) {
  check(what, gc_rms_norm(in<void>(), nullptr, in<void>(), &rows, 1, hidden, 1e-6f, t, nullptr, list(), yt, nullptr, nullptr), least);
}

void pack(const char* what, int64_t rows, size_t n, gc_dtype t, uint64_t least) {
  check(what, gc_mx8_pack(in<void>(), &rows, 1, n, t, list(), nullptr), least);
  check(what, gc_mx8_unpack(in<void>(), &rows, 1, n, t, list(), nullptr), least);
}

// Launches of a forward without checkpoint: 2 streamed (each reads an expert's weights again
// for every 16 or 8 of its rows), 3 in tiles.
void forward_launches(int64_t rows, int E, size_t hidden, size_t inter, size_t want) {
  const size_t need = gc_moe_ffn_scratch_bytes(&rows, 1, E, hidden, inter, GC_BF16, 0);
  gc_moe_ffn(in<void>(), GC_BF16, &rows, static_cast<int64_t*>(buf()), 1, E, hidden, inter, in<void>(), in<void>(), in<void>(), nullptr,
             GC_BF16, list(), buf(), need, nullptr);
  const size_t got = g_launches.size();
  g_failures += got != want;
  std::printf("experts' forward, %lld rows over %d: %zu launches: %s\n", static_cast<long long>(rows), E, got, got == want ? "ok" : "FAILED");
  g_launches.clear();
}

void experts(const char* what, int64_t rows, int E, size_t hidden, size_t inter, gc_dtype xt, bool backward, uint64_t least) {
  const size_t need = gc_moe_ffn_scratch_bytes(&rows, 1, E, hidden, inter, xt, backward);
  const int64_t* splits = static_cast<int64_t*>(buf());
  if (backward)
    check(what, gc_moe_ffn_backward(in<void>(), in<void>(), xt, in<void>(), GC_BF16, &rows, splits, 1, E, hidden, inter, in<void>(),
                                    in<void>(), in<void>(), list(), list(), list(), list(), GC_BF16, buf(), need, nullptr), least);
  else
    check(what, gc_moe_ffn(in<void>(), xt, &rows, splits, 1, E, hidden, inter, in<void>(), in<void>(), in<void>(), nullptr, GC_BF16,
                           list(), buf(), need, nullptr), least);
}

}  // namespace

extern "C" hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
  g_launches.push_back({grid, block});
  return hipSuccess;
}

int main() {
  g_lists.reserve(4096);
  const int64_t most = (int64_t(1) << 31) - 1;
  pack("8-bit rows, 2^26 + 3 of 32", (int64_t(1) << 26) + 3, 32, GC_BF16, (1 << 24) + 1);
  pack("8-bit rows, 2^31 - 1 of 1", most, 1, GC_FP32, 1 << 29);
  pack("8-bit rows, 2^24 + 1 of 4104", (int64_t(1) << 24) + 1, 4104, GC_BF16, (1 << 24) + 1);
  norm("norm, 2^26 + 3 of 8", (int64_t(1) << 26) + 3, 8, GC_BF16, GC_BF16, (1 << 24) + 1);
  norm("norm, 2^31 - 1 of 1 to 8-bit rows", most, 1, GC_FP32, GC_MX8, 1 << 29);
  norm("norm, 2^24 + 1 of 1032", (int64_t(1) << 24) + 1, 1032, GC_BF16, GC_BF16, (1 << 24) + 1);
  norm("norm, 2^24 + 1 of 16392", (int64_t(1) << 24) + 1, 16392, GC_BF16, GC_BF16, (1 << 24) + 1);
  {
    const int64_t rows = 1;
    const size_t H = size_t(1) << 31, need = gc_rms_norm_backward_scratch_bytes(&rows, 1, H);
    check("norm backward, one row of 2^31",
          gc_rms_norm_backward(in<void>(), nullptr, in<void>(), in<void>(), in<float>(), &rows, 1, H, GC_BF16, list(),
                               reinterpret_cast<float* const*>(list()), buf(), need, nullptr), 1 + (1 << 25));
  }
  {
    const int64_t tokens = (int64_t(1) << 27) + 5, rows = 7;
    check("combine gradient, 2^27 + 5 tokens of 257",
          gc_moe_combine_backward(in<void>(), in<void>(), &rows, in<int32_t>(), in<float>(), &tokens, 1, 1, 257, GC_BF16, list(),
                                  reinterpret_cast<float* const*>(list()), nullptr), (1 << 25) + 2);
  }
  experts("experts, 5 rows, 1024 of 8 x 2^20", 5, 1024, 8, size_t(1) << 20, GC_BF16, false, 500);
  experts("experts' backward, 1024 of 8 x 2^20", 5, 1024, 8, size_t(1) << 20, GC_BF16, true, 1000);
  experts("experts' backward, 8192 of 8 x 2^16", 9000, 8192, 8, size_t(1) << 16, GC_BF16, true, 1000);
  experts("experts, 5 rows, 1024 of 2^20 x 8", 5, 1024, size_t(1) << 20, 8, GC_BF16, false, 200);
  experts("experts, streamed, 64 of 8 x 2^20", 5, 64, 8, size_t(1) << 20, GC_BF16, false, 64 * 8192);
  experts("experts, 2^26 + 5 8-bit rows of 8", (int64_t(1) << 26) + 5, 1, 8, 8, GC_MX8, false, (1 << 24) + 2);
  experts("experts' backward, 2^26 + 5 8-bit rows", (int64_t(1) << 26) + 5, 1, 8, 8, GC_MX8, true, (1 << 24) + 2);
  // one expert may get every row, so the streamed form is for few rows in all
  forward_launches(8000, 1024, 2048, 1024, 3);
  forward_launches(500, 64, 2048, 1024, 3);
  forward_launches(33, 64, 2048, 1024, 3);
  forward_launches(8, 256, 2048, 1024, 3);
  forward_launches(32, 64, 2048, 1024, 2);
  forward_launches(1, 8, 4096, 11008, 2);
  std::printf("%d failures\n", g_failures);
  return g_failures != 0;
}
