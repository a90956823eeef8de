// Seeded argument fuzz of the ABI of embedding, dropout and log probabilities
// (api_token.cpp), built for the host with AddressSanitizer and
// UndefinedBehaviorSanitizer against token_stubs.cpp.  Host arrays have exactly the length the contract names;
// arguments are drawn mostly valid with a few perturbed.  Checked: a known
// status; a refused call launches nothing; launches stay inside the declared
// buffers; every entry point is both accepted and refused.
//
// usage: token_fuzz [iterations] [seed]
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

template <class T>
T* const* out(const std::vector<T*>& v) { return const_cast<T* const*>(v.data()); }

void one(uint64_t) {
  g_at = 1ull << 36;
  const int N = ranks(), n = N > 0 ? N : 0;
  const long before = stub::launches();
  const gc_dtype t = type(coin(0.5) ? GC_BF16 : GC_FP32), wt = type(coin(0.5) ? GC_BF16 : GC_FP32);
  const uint64_t es = t == GC_BF16 ? 2 : 4, ws = wt == GC_BF16 ? 2 : 4;
  const float scale = coin(0.02) ? 0.0f / 0.0f : coin(0.02) ? -1.0f : coin(0.02) ? 3e38f : 1.5f;
  switch (rnd(5)) {
    case 0: {
      const size_t v = coin(0.1) ? 1 + rnd(1u << 22) : dim(1, 3000), h = dim(1, 200);
      const auto tok = counts(N, 40);
      const bool sane = v < (1ull << 23) && h < (1ull << 20);
      const auto w = bufs(n, std::vector<uint64_t>(n, sane ? v * h * es : 0)), o = bufs(n, scaled(tok, h * es));
      const auto ids = bufs<int32_t>(n, scaled(tok, 4));
      check("gc_embedding", gc_embedding(in(w), in(ids), tok.data(), N, v, h, scale, t, out(o), nullptr), before);
      break;
    }
    case 1: {
      const size_t v = coin(0.1) ? 1 + rnd(1u << 22) : dim(1, 3000), h = dim(1, 200);
      const auto tok = counts(N, coin(0.2) ? 9000 : 40);
      const bool sane = v < (1ull << 23) && h < (1ull << 20);
      const auto g = bufs(n, scaled(tok, h * es)), dw = bufs(n, std::vector<uint64_t>(n, sane ? v * h * ws : 0));
      const auto ids = bufs<int32_t>(n, scaled(tok, 4));
      const size_t need = n ? gc_embedding_backward_scratch_bytes(tok.data(), N, v, h) : 0;
      void* sc = buf(need < (1ull << 40) ? need : 0);
      check("gc_embedding_backward",
            gc_embedding_backward(in(g), in(ids), tok.data(), N, v, h, scale, t, out(dw), wt, coin(0.5), sc, coin(0.02) ? need - 1 : need, nullptr),
            before);
      break;
    }
    case 2: {
      const auto c = counts(N, 5000);
      std::vector<uint64_t> bytes;   // element counts may be as large as a buffer
      for (int64_t k : c) bytes.push_back(k > 0 && k <= (int64_t(1) << 40) ? k * es : 0);
      const auto x = bufs(n, bytes), res = bufs(n, bytes), y = bufs(n, bytes);
      const uint64_t* step = static_cast<uint64_t*>(coin(0.5) ? nullptr : buf(8));
      const auto& o = coin(0.2) ? x : coin(0.2) ? res : y;
      check("gc_dropout",
            gc_dropout(in(x), coin(0.4) ? nullptr : in(res), c.data(), N, coin(0.03) ? 1.5f : 0.1f, g_rng(), g_rng(), step, t, out(o), nullptr),
            before);
      break;
    }
    default: {
      const size_t v = coin(0.3) ? dim(1, 200000) : dim(1, 3000), pad = coin(0.5) ? rnd(70) : 0;
      const size_t stride = coin(0.02) ? v - 1 : v + pad;
      const int top = coin(0.03) ? static_cast<int>(rnd(80)) - 5 : coin(0.5) ? 0 : 1 + static_cast<int>(rnd(64));
      const auto tok = counts(N, 40);
      const uint64_t k = top > 0 ? top : 0, row = stride < (1ull << 30) ? stride * es : 0;
      const auto x = bufs(n, scaled(tok, row)), dx = bufs(n, scaled(tok, row));
      const auto ids = bufs<int32_t>(n, scaled(tok, 4)), ti = bufs<int32_t>(n, scaled(tok, 4 * k));
      const auto lp = bufs<float>(n, scaled(tok, 4)), h = bufs<float>(n, scaled(tok, 4)), lse = bufs<float>(n, scaled(tok, 4)),
                 a = bufs<float>(n, scaled(tok, 4)), b = bufs<float>(n, scaled(tok, 4)), tl = bufs<float>(n, scaled(tok, 4 * k));
      const bool given = coin(0.8), grad = given && coin(0.4), ent = coin(0.5);
      const auto& o = coin(0.3) ? x : dx;
      if (coin(0.4)) {
        check("gc_token_logprob_backward",
              gc_token_logprob_backward(in(x), coin(0.02) ? nullptr : in(ids), in(lse), ent || coin(0.5) ? in(h) : nullptr, in(a),
                                        ent ? in(b) : nullptr, tok.data(), N, v, stride, scale, t, out(o), nullptr),
              before);
        break;
      }
      const size_t need = n ? gc_token_logprob_scratch_bytes(tok.data(), N, v, top) : 0;
      void* sc = buf(need < (1ull << 40) ? need : 0);
      check("gc_token_logprob",
            gc_token_logprob(in(x), given ? in(ids) : nullptr, tok.data(), N, v, stride, scale, t,
                             given || coin(0.02) ? out(lp) : nullptr, coin(0.5) ? out(h) : nullptr, coin(0.5) ? out(lse) : nullptr, top,
                             out(ti), out(tl), grad || coin(0.02) ? in(a) : nullptr, grad && ent ? in(b) : nullptr, grad ? out(o) : nullptr, sc,
                             coin(0.02) ? need - 1 : need, nullptr),
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
