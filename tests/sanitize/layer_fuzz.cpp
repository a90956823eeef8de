// Seeded argument fuzz of the layer operators' ABI (api_layer.cpp), built for
// the host with AddressSanitizer and UndefinedBehaviorSanitizer against
// layer_stubs.cpp.  Host arrays have exactly the length the contract names;
// arguments are drawn mostly valid with a few perturbed.  Checked: a known
// status; a refused call launches nothing; launches stay inside the declared
// buffers; every entry point is both accepted and refused.
//
// usage: layer_fuzz [iterations] [seed]
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <string>
#include <vector>

#include "gc.h"
#include "gc_internal.h"
#include "stubs.h"

namespace {

std::mt19937_64 g_rng;
int g_failures = 0;
struct Tally {
  long ok = 0, refused = 0;
};
std::map<std::string, Tally> g_tally;

uint64_t rnd(uint64_t n) { return n ? g_rng() % n : 0; }
bool coin(double p) { return (g_rng() >> 11) * 0x1p-53 < p; }

uint64_t g_at = 0;
// A stand-in buffer of `bytes`, now and then null, misaligned, on top of the last one or near the end of the address space.
void* buf(uint64_t bytes) {
  if (coin(0.003)) return nullptr;
  uint64_t p = g_at;
  if (coin(0.003)) p -= 4096;                       // over the one before
  else if (coin(0.003)) p = UINT64_MAX - rnd(4096);
  else g_at += (bytes + 8191) / 4096 * 4096;
  if (coin(0.004)) p += 1 + rnd(15);
  stub::declare(reinterpret_cast<void*>(p), bytes);
  return reinterpret_cast<void*>(p);
}
template <class T = void>
std::vector<T*> bufs(int n, const std::vector<uint64_t>& bytes) {
  std::vector<T*> v(n > 0 ? n : 0);
  for (int i = 0; i < n; ++i) v[i] = static_cast<T*>(buf(bytes[i]));
  return v;
}
template <class T>
auto in(const std::vector<T*>& v) { return const_cast<const T* const*>(v.data()); }

void check(const char* what, gc_status s, long before) {
  if (s < GC_OK || s > GC_ERR_NO_MEMORY) ++g_failures, std::fprintf(stderr, "%s: status %d\n", what, s);
  if (s != GC_OK && stub::launches() != before) ++g_failures, std::fprintf(stderr, "%s: refused after a launch\n", what);
  (s == GC_OK ? g_tally[what].ok : g_tally[what].refused)++;
}

int ranks() { return coin(0.02) ? static_cast<int>(rnd(80)) - 5 : 1 + static_cast<int>(rnd(10)); }
gc_dtype type(gc_dtype usual) { return coin(0.05) ? static_cast<gc_dtype>(rnd(4)) : usual; }
size_t dim(size_t step, size_t most) { return coin(0.03) ? g_rng() >> rnd(64) : step * (1 + rnd(most)); }
std::vector<int64_t> counts(int n, int64_t most) {
  std::vector<int64_t> v(n > 0 ? n : 0);
  for (auto& c : v) c = coin(0.01) ? static_cast<int64_t>(g_rng() >> rnd(64)) - 2 : static_cast<int64_t>(rnd(most));
  return v;
}
std::vector<uint64_t> scaled(const std::vector<int64_t>& c, uint64_t b) {
  std::vector<uint64_t> v;
  for (int64_t x : c) v.push_back(x > 0 && b < (1ull << 40) && static_cast<uint64_t>(x) < (1ull << 23) ? x * b : 0);
  return v;
}

void one(uint64_t) {
  g_at = 1ull << 36;
  const int N = ranks(), n = N > 0 ? N : 0;
  const long before = stub::launches();
  const gc_dtype t = type(coin(0.5) ? GC_BF16 : GC_FP32);
  const uint64_t es = t == GC_BF16 ? 2 : 4;
  switch (rnd(6)) {
    case 0:
    case 1: {
      const size_t k = dim(1, 200);
      const auto rows = counts(N, 20);
      const uint64_t r8 = k < (1ull << 32) ? gci::mx8_row_bytes(k) : 0;
      const auto a = bufs(n, scaled(rows, coin(0.5) ? r8 : k * es)), b = bufs(n, scaled(rows, std::max<uint64_t>(r8, k * es)));
      const auto dense = bufs(n, scaled(rows, k * es)), packed = bufs(n, scaled(rows, r8));
      (void)a, (void)b;
      if (coin(0.5)) check("gc_mx8_pack", gc_mx8_pack(in(dense), rows.data(), N, k, t, const_cast<void* const*>(packed.data()), nullptr), before);
      else check("gc_mx8_unpack", gc_mx8_unpack(in(packed), rows.data(), N, k, t, const_cast<void* const*>(dense.data()), nullptr), before);
      break;
    }
    case 2: {
      const size_t h = dim(1, 200);
      const auto tok = counts(N, 20);
      const auto rows = scaled(tok, h * es);
      std::vector<uint64_t> w(n, h < (1ull << 32) ? h * es : 0);
      const gc_dtype yt = coin(0.3) ? GC_MX8 : type(t);
      const auto x = bufs(n, rows), res = bufs(n, rows), wt = bufs(n, w), sum = bufs(n, rows);
      const auto y = bufs(n, scaled(tok, yt == GC_MX8 && h < (1ull << 32) ? gci::mx8_row_bytes(h) : h * es));
      const auto rs = bufs<float>(n, scaled(tok, 4));
      void* const* so = coin(0.3) ? nullptr : coin(0.3) ? const_cast<void* const*>(x.data()) : const_cast<void* const*>(sum.data());
      check("gc_rms_norm",
            gc_rms_norm(in(x), coin(0.3) ? nullptr : in(res), in(wt), tok.data(), N, h, coin(0.02) ? -1.0f : 1e-6f, t, so,
                        const_cast<void* const*>(y.data()), yt, coin(0.3) ? nullptr : const_cast<float* const*>(rs.data()), nullptr),
            before);
      break;
    }
    case 3: {
      const size_t h = dim(1, 200);
      const auto tok = counts(N, 40);
      const auto rows = scaled(tok, h * es);
      std::vector<uint64_t> w(n, h < (1ull << 32) ? h * es : 0), w4(n, h < (1ull << 32) ? h * 4 : 0);
      const size_t need = n ? gc_rms_norm_backward_scratch_bytes(tok.data(), N, h) : 0;
      const auto dy = bufs(n, rows), ds = bufs(n, rows), s = bufs(n, rows), wt = bufs(n, w), dx = bufs(n, rows);
      const auto rs = bufs<float>(n, scaled(tok, 4)), dw = bufs<float>(n, w4);
      void* sc = buf(need < (1ull << 40) ? need : 0);
      void* const* out = coin(0.3) ? const_cast<void* const*>(dy.data()) : const_cast<void* const*>(dx.data());
      check("gc_rms_norm_backward",
            gc_rms_norm_backward(in(dy), coin(0.4) ? nullptr : in(ds), in(s), in(wt), in(rs), tok.data(), N, h, t, out,
                                 const_cast<float* const*>(dw.data()), sc, coin(0.02) ? need - 1 : need, nullptr),
            before);
      break;
    }
    case 4: {
      const size_t h = dim(1, 200);
      const int K = coin(0.03) ? static_cast<int>(rnd(12)) - 1 : 1 + static_cast<int>(rnd(8));
      const auto tok = counts(N, 20), er = counts(N, 40);
      const uint64_t k = K > 0 ? K : 0;
      const auto g = bufs(n, scaled(tok, h * es)), y = bufs(n, scaled(er, h * es)), dy = bufs(n, scaled(er, h * es));
      const auto dest = bufs<int32_t>(n, scaled(tok, k * 8));
      const auto w = bufs<float>(n, scaled(tok, k * 4)), dw = bufs<float>(n, scaled(tok, k * 4));
      check("gc_moe_combine_backward",
            gc_moe_combine_backward(in(g), in(y), er.data(), in(dest), in(w), tok.data(), N, K, h, t,
                                    const_cast<void* const*>(dy.data()), const_cast<float* const*>(dw.data()), nullptr),
            before);
      break;
    }
    default: {
      const size_t h = dim(8, 40), f = coin(0.5) ? dim(32, 10) : dim(8, 40);
      const int E = coin(0.02) ? static_cast<int>(rnd(20000)) - 3 : 1 + static_cast<int>(rnd(6));
      const auto rows = counts(N, 600);
      const gc_dtype xt = type(coin(0.3) ? GC_MX8 : GC_BF16), st = type(coin(0.5) ? GC_MX8 : GC_BF16), wt = type(coin(0.5) ? GC_FP32 : GC_BF16);
      const bool sane = h < (1ull << 24) && f < (1ull << 24) && E > 0 && E < 10000;
      const uint64_t w = sane ? static_cast<uint64_t>(E) * h * f * 2 : 0;
      const bool back = coin(0.5);
      const size_t need = n ? gc_moe_ffn_scratch_bytes(rows.data(), N, E, h, f, xt, back) : 0;
      const std::vector<uint64_t> ws(n, w), dws(n, wt == GC_FP32 ? 2 * w : w);
      const auto x = bufs(n, scaled(rows, sane && xt == GC_MX8 ? gci::mx8_row_bytes(h) : h * 2));
      const auto sv = bufs(n, scaled(rows, sane && st == GC_MX8 ? gci::mx8_row_bytes(2 * f) : f * 4));
      const auto y = bufs(n, scaled(rows, h * 2)), dy = bufs(n, scaled(rows, h * 2));
      const auto wg = bufs(n, ws), wu = bufs(n, ws), wd = bufs(n, ws), dg = bufs(n, dws), du = bufs(n, dws), dd = bufs(n, dws);
      const int64_t* splits = static_cast<int64_t*>(buf(sane && n ? static_cast<uint64_t>(n) * n * E * 8 : 0));
      void* sc = buf(need < (1ull << 40) ? need : 0);
      const size_t given = coin(0.02) ? need - 1 : need;
      const bool keep = coin(0.7);
      if (back)
        check("gc_moe_ffn_backward",
              gc_moe_ffn_backward(in(dy), in(x), xt, keep ? in(sv) : nullptr, st, rows.data(), splits, N, E, h, f, in(wg), in(wu),
                                  in(wd), const_cast<void* const*>(y.data()), const_cast<void* const*>(dg.data()),
                                  const_cast<void* const*>(du.data()), const_cast<void* const*>(dd.data()), wt, sc, given, nullptr),
              before);
      else
        check("gc_moe_ffn",
              gc_moe_ffn(in(x), xt, rows.data(), splits, N, E, h, f, in(wg), in(wu), in(wd),
                         keep ? const_cast<void* const*>(sv.data()) : nullptr, st, const_cast<void* const*>(y.data()), sc, given,
                         nullptr),
              before);
    }
  }
}

}  // namespace

int main(int argc, char** argv) {
  const uint64_t iters = argc > 1 ? std::strtoull(argv[1], nullptr, 10) : 20000;
  g_rng.seed(argc > 2 ? std::strtoull(argv[2], nullptr, 10) : 1);
  for (uint64_t i = 0; i < iters; ++i) {
    stub::reset();
    one(i);
  }
  if (stub::violations()) ++g_failures, std::fprintf(stderr, "%ld launches left the declared memory\n", stub::violations());
  for (const auto& t : g_tally) {
    std::printf("%-26s ok %6ld  refused %6ld\n", t.first.c_str(), t.second.ok, t.second.refused);
    if (!t.second.ok || !t.second.refused) ++g_failures;
  }
  std::printf("%ld launches, %d failures\n", stub::launches(), g_failures);
  return g_failures ? 1 : 0;
}
