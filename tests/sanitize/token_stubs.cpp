// Host-only stand-ins for the launchers of embedding, dropout and log
// probabilities, for the sanitizer build of api_token.cpp: every byte range a
// launch would touch must lie inside a buffer the harness declared with the
// extent the contract gives.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "gc_internal.h"
#include "stubs.h"

namespace stub {

uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

namespace {
struct Buf {
  uint64_t lo, hi;
};
std::vector<Buf> g_bufs;
long g_launches = 0, g_bad = 0;

void need(const void* p, uint64_t bytes, const char* what) {
  if (!bytes) return;
  for (const Buf& b : g_bufs)
    if (b.lo <= addr(p) && addr(p) <= b.hi && bytes <= b.hi - addr(p)) return;
  std::fprintf(stderr, "launch touches undeclared memory: %s\n", what);
  ++g_bad;
}
void must(bool ok, const char* what) {
  if (!ok) std::fprintf(stderr, "%s\n", what), ++g_bad;
}
}  // namespace

void reset() { g_bufs.clear(); }
void declare(const void* p, uint64_t bytes) {
  if (p && bytes) g_bufs.push_back(Buf{addr(p), addr(p) + bytes});
}
long launches() { return g_launches; }
long violations() { return g_bad; }

}  // namespace stub

namespace gci {

using stub::must;
using stub::need;

gc_status launch_embedding(const EmbeddingCall& c) {
  const uint64_t row = c.hidden * elem_bytes(c.t);
  for (int r = 0; r < c.nranks; ++r) {
    const uint64_t n = c.tokens[r];
    if (n) need(c.w[r], c.vocab * row, "embedding weight");
    need(c.ids[r], n * 4, "embedding tokens");
    need(c.out[r], n * row, "embedding rows");
  }
  ++stub::g_launches;
  return GC_OK;
}

gc_status launch_embedding_backward(const EmbeddingBackwardCall& c) {
  const EmbeddingGeom& g = c.geom;
  uint64_t chunks = 0, runs = 0, tokens = 0;
  for (int r = 0; r < c.nranks; ++r) {
    const uint64_t n = c.tokens[r];
    need(c.dout[r], n * c.hidden * elem_bytes(c.t), "embedding gradient rows");
    need(c.ids[r], n * 4, "embedding tokens");
    need(c.dw[r], c.vocab * c.hidden * elem_bytes(c.dw_t), "embedding weight gradient");
    chunks += std::max<uint64_t>(1, (n + g.chunk - 1) / g.chunk);
    runs += (n + g.run - 1) / g.run;
    tokens += n;
  }
  // the areas of the scratch follow one another and hold what the kernels put there
  must(g.chunk % 512 == 0 && chunks == static_cast<uint64_t>(g.chunks), "sorting pieces");
  must(g.low_bits >= 1 && g.low_bits <= kEmbeddingDigit && g.bits - g.low_bits <= kEmbeddingDigit && c.vocab <= uint64_t(1) << g.bits,
       "digits of the id");
  must(g.low_bits == g.bits || g.keys - g.pairs >= tokens * 8, "pairs");
  must(g.perm - g.keys >= tokens * 4 && g.counts - g.perm >= tokens * 4, "sorted lists");
  must(g.valid - g.counts >= chunks * 4 << std::max(g.low_bits, g.bits - g.low_bits), "digit counts");
  must(g.present - g.valid >= 4u * c.nranks, "valid counts");
  must(g.present_row >= c.vocab && g.present_row % 16 == 0 && g.long_rows - g.present >= c.nranks * g.present_row, "map of tokens");
  must(g.partial - g.long_rows >= (runs + 1) * 4, "list of long rows");
  must(embedding_pitch(c.hidden) >= c.hidden && g.bytes - g.partial >= runs * 2 * embedding_pitch(c.hidden) * 4, "partial rows");
  for (uint64_t at : {g.pairs, g.keys, g.perm, g.counts, g.valid, g.present, g.long_rows, g.partial}) must(at % 256 == 0, "alignment");
  need(c.scratch, g.bytes, "embedding scratch");
  ++stub::g_launches;
  return GC_OK;
}

gc_status launch_dropout(const DropoutCall& c) {
  for (int r = 0; r < c.nranks; ++r) {
    const uint64_t bytes = static_cast<uint64_t>(c.counts[r]) * elem_bytes(c.t);
    need(c.x[r], bytes, "dropout x");
    if (c.res) need(c.res[r], bytes, "dropout residual");
    need(c.y[r], bytes, "dropout y");
  }
  if (c.step) need(c.step, 8, "dropout step");
  must(c.drop <= 65536, "dropout threshold");
  ++stub::g_launches;
  return GC_OK;
}

static gc_status logprob_like(const LogprobCall& c, bool backward) {
  uint64_t rows = 0;
  for (int r = 0; r < c.nranks; ++r) {
    const uint64_t n = c.tokens[r], bytes = n * c.stride * elem_bytes(c.t);
    rows += n;
    need(c.logits[r], bytes, "logits");
    if (c.targets) need(c.targets[r], n * 4, "targets");
    for (float* const* p : {c.logprob, c.entropy, c.lse})
      if (p) need(p[r], n * 4, "row numbers");
    for (const float* const* p : {c.dlogprob, c.dentropy})
      if (p) need(p[r], n * 4, "gradients of row numbers");
    if (c.top) need(c.top_ids[r], n * 4 * c.top, "alternatives"), need(c.top_logprob[r], n * 4 * c.top, "their log probabilities");
    if (c.dlogits) need(c.dlogits[r], bytes, "gradient of logits");
  }
  must(c.parts >= 1 && c.parts <= kLogprobParts, "parts of a row");
  must(!backward || (c.dlogits && c.dlogprob && c.targets && c.lse && !c.dentropy == !c.entropy), "what the gradient needs");
  if (!backward && c.parts > 1) need(c.scratch, rows * c.parts * (16 + 8 * static_cast<uint64_t>(c.top)), "parts' scratch");
  ++stub::g_launches;
  return GC_OK;
}
gc_status launch_token_logprob(const LogprobCall& c) { return logprob_like(c, false); }
gc_status launch_token_logprob_backward(const LogprobCall& c) { return logprob_like(c, true); }

}  // namespace gci
