// C ABI of the two ends of a training step: token embedding and its gradient,
// dropout, token log probabilities and their gradient.  Argument validation and
// aliasing rules, then the launches.  Every check runs before anything is
// enqueued, and nothing here allocates.

#include <cmath>

#include "api_checks.h"

namespace {

using namespace gca;

constexpr size_t kMaxVocab = size_t(1) << 22;   // of an embedding: two digits of gci::kEmbeddingDigit bits
constexpr int kMaxTop = 64;
constexpr float kMaxScale = 0x1p64f;            // of logits: times log2(e) it stays a number

gc_status check_row_type(gc_dtype t) {
  if (t != GC_MX8 && !valid_dtype(t)) return GC_ERR_INVALID_ARG;
  return row_type(t) ? GC_OK : GC_ERR_UNSUPPORTED;
}

template <class T>
const void* const* any(T* const* p) { return reinterpret_cast<const void* const*>(p); }

uint64_t up256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

}  // namespace

// ------------------------------------------------------------- embedding

namespace {

gc_status embedding_sizes(const int64_t* ntokens, int nranks, size_t vocab, size_t hidden) {
  GC_TRY(check_rows(ntokens, nranks));
  if (vocab == 0 || hidden == 0) return GC_ERR_INVALID_ARG;
  return vocab > kMaxVocab || hidden > kMaxRow ? GC_ERR_UNSUPPORTED : GC_OK;
}

}  // namespace

extern "C" gc_status gc_embedding(const void* const* weight, const int32_t* const* tokens, const int64_t* ntokens,
                                  int nranks, size_t vocab, size_t hidden, float scale, gc_dtype t, void* const* out,
                                  hipStream_t stream) {
  GC_TRY(embedding_sizes(ntokens, nranks, vocab, hidden));
  if (!std::isfinite(scale)) return GC_ERR_INVALID_ARG;
  GC_TRY(check_row_type(t));
  const size_t es = elem_bytes(t);
  const uint64_t row = hidden * es;
  Buffers b;
  b.add(weight, nranks, es, [&](int r) { return ntokens[r] ? vocab * row : 0; }, false);
  b.add(any(tokens), nranks, 4, [&](int r) { return static_cast<uint64_t>(ntokens[r]) * 4; }, false);
  b.add(any(out), nranks, es, [&](int r) { return static_cast<uint64_t>(ntokens[r]) * row; }, true);
  GC_TRY(b.check());
  return gci::launch_embedding({weight, tokens, ntokens, nranks, vocab, hidden, scale, t, out, stream});
}

// Ranks of at most 2048 tokens are sorted by one workgroup each, in one launch (a gradient of 2048 x 256 takes 26 us so,
// 28 in pieces; 4096 x 256 35 and 31); longer ones by a workgroup per 1024 tokens (two of each lane), more where a rank
// would make over 256 pieces: every piece reads the counts of all the others.  A group of lanes sums a run of 8 sorted
// tokens where they are few, for more groups (517 x 1000 fp32: 16 us, 28 with 64), and of up to 64 where those are a
// thousand, for fewer partial sums (8 x 16384 x 4096 bf16, frequent tokens: 584 us, 599 with 8; none frequent: 642, 604).
gci::EmbeddingGeom gci::embedding_geom(const int64_t* tokens, int nranks, uint64_t vocab, uint64_t hidden) {
  gci::EmbeddingGeom g;
  int64_t most = 0;
  for (int r = 0; r < nranks; ++r) {
    g.tokens += tokens[r];
    most = std::max(most, tokens[r]);
  }
  const auto up512 = [](int64_t x) { return (std::max<int64_t>(x, 1) + 511) / 512 * 512; };
  g.chunk = static_cast<int32_t>(most <= 2048 ? up512(most) : std::max<int64_t>(1024, up512(most / 256)));
  for (int r = 0; r < nranks; ++r) g.chunks += static_cast<int32_t>(std::max<int64_t>(1, (tokens[r] + g.chunk - 1) / g.chunk));
  g.bits = 1;
  while (vocab > uint64_t(1) << g.bits) ++g.bits;
  g.low_bits = g.bits <= kEmbeddingDigit ? g.bits : (g.bits + 1) / 2;
  g.run = 8;
  while (g.run < 64 && g.tokens / g.run >= 1024) g.run *= 2;
  uint64_t runs = 0;
  for (int r = 0; r < nranks; ++r) runs += static_cast<uint64_t>(tokens[r] + g.run - 1) / g.run;
  const uint64_t n = static_cast<uint64_t>(g.tokens);
  g.keys = g.pairs + (g.low_bits < g.bits ? up256(n * 8) : 0);
  g.perm = g.keys + up256(n * 4);
  g.counts = g.perm + up256(n * 4);
  g.valid = g.counts + up256(static_cast<uint64_t>(g.chunks) * 4 << g.low_bits);
  g.present = g.valid + up256(static_cast<uint64_t>(nranks) * 4);
  g.present_row = (vocab + 15) / 16 * 16;
  g.long_rows = g.present + up256(nranks * g.present_row);
  g.partial = g.long_rows + up256((runs + 1) * 4);
  g.bytes = g.partial + up256(runs * 2 * embedding_pitch(hidden) * 4);
  return g;
}

extern "C" size_t gc_embedding_backward_scratch_bytes(const int64_t* ntokens, int nranks, size_t vocab, size_t hidden) {
  if (embedding_sizes(ntokens, nranks, vocab, hidden) != GC_OK) return 0;
  return gci::embedding_geom(ntokens, nranks, vocab, hidden).bytes;
}

extern "C" gc_status gc_embedding_backward(const void* const* dout, const int32_t* const* tokens,
                                           const int64_t* ntokens, int nranks, size_t vocab, size_t hidden, float scale,
                                           gc_dtype t, void* const* dweight, gc_dtype dw_t, int accumulate,
                                           void* scratch, size_t scratch_bytes, hipStream_t stream) {
  GC_TRY(embedding_sizes(ntokens, nranks, vocab, hidden));
  if (!std::isfinite(scale)) return GC_ERR_INVALID_ARG;
  GC_TRY(check_row_type(t));
  GC_TRY(check_row_type(dw_t));
  const gci::EmbeddingGeom g = gci::embedding_geom(ntokens, nranks, vocab, hidden);
  if (scratch_bytes < g.bytes) return GC_ERR_INVALID_ARG;
  const size_t es = elem_bytes(t), ws = elem_bytes(dw_t);
  Buffers b;
  b.add(dout, nranks, es, [&](int r) { return static_cast<uint64_t>(ntokens[r]) * hidden * es; }, false);
  b.add(any(tokens), nranks, 4, [&](int r) { return static_cast<uint64_t>(ntokens[r]) * 4; }, false);
  b.add(any(dweight), nranks, ws, [&](int) { return static_cast<uint64_t>(vocab) * hidden * ws; }, true);
  b.one(scratch, 256, g.bytes, true);
  GC_TRY(b.check());
  return gci::launch_embedding_backward(
      {dout, tokens, ntokens, nranks, vocab, hidden, scale, t, dweight, dw_t, accumulate != 0, scratch, g, stream});
}

// ------------------------------------------------------------- dropout

extern "C" gc_status gc_dropout(const void* const* x, const void* const* residual, const int64_t* counts, int nranks,
                                float p, uint64_t seed, uint64_t offset, const uint64_t* step, gc_dtype t,
                                void* const* y, hipStream_t stream) {
  GC_TRY(check_ranks(nranks));
  if (!counts || !(p >= 0.0f && p <= 1.0f)) return GC_ERR_INVALID_ARG;
  GC_TRY(check_row_type(t));
  const size_t es = elem_bytes(t);
  for (int r = 0; r < nranks; ++r)
    if (counts[r] < 0 || static_cast<uint64_t>(counts[r]) > kMaxExtent) return GC_ERR_INVALID_ARG;
  const auto bytes = [&](int r) { return static_cast<uint64_t>(counts[r]) * es; };
  Buffers b;
  b.add(x, nranks, es, [&](int r) { return same(y, x, r) ? 0 : bytes(r); }, false);
  if (residual) b.add(residual, nranks, es, [&](int r) { return same(y, residual, r) ? 0 : bytes(r); }, false);
  b.add(any(y), nranks, es, bytes, true);
  if (step) b.one(step, 8, 8, false);
  GC_TRY(b.check());
  const uint32_t drop = static_cast<uint32_t>(std::floor(static_cast<double>(p) * 65536.0 + 0.5));
  const float scale = drop < 65536 ? static_cast<float>(65536.0 / (65536 - drop)) : 0.0f;
  return gci::launch_dropout({x, residual, counts, nranks, drop, scale, seed, offset, step, t, y, stream});
}

// ------------------------------------------------------------- log probabilities

namespace {

gc_status logprob_sizes(const int64_t* ntokens, int nranks, size_t vocab, int top) {
  GC_TRY(check_rows(ntokens, nranks));
  if (vocab == 0 || top < 0) return GC_ERR_INVALID_ARG;
  if (vocab > kMaxRow || top > kMaxTop) return GC_ERR_UNSUPPORTED;
  return static_cast<size_t>(top) > vocab ? GC_ERR_INVALID_ARG : GC_OK;
}

// What both directions check.
gc_status logprob_check(const gci::LogprobCall& c, Buffers& b) {
  if (c.stride < c.vocab || !(c.scale > 0.0f && c.scale <= kMaxScale)) return GC_ERR_INVALID_ARG;
  if (c.stride > kMaxRow) return GC_ERR_UNSUPPORTED;
  GC_TRY(check_row_type(c.t));
  const size_t es = elem_bytes(c.t);
  const uint64_t row = c.stride * es;
  const auto rows = [&c](uint64_t bytes) { return [&c, bytes](int r) { return static_cast<uint64_t>(c.tokens[r]) * bytes; }; };
  b.add(c.logits, c.nranks, es,
        [&](int r) { return same(c.dlogits, c.logits, r) ? 0 : static_cast<uint64_t>(c.tokens[r]) * row; }, false);
  if (c.targets) b.add(any(c.targets), c.nranks, 4, rows(4), false);
  if (c.dlogits) {
    b.add(any(c.dlogits), c.nranks, es, rows(row), true);
    b.add(any(c.dlogprob), c.nranks, 4, rows(4), false);
    if (c.dentropy) b.add(any(c.dentropy), c.nranks, 4, rows(4), false);
  }
  return GC_OK;
}

}  // namespace

namespace {

// A workgroup per row leaves most of the chip idle where there are few rows.  Few long ones are cut into parts of 8192
// logits or more, 256 parts in all, for a second launch to join; one row of 32000 with 20 alternatives takes 12 us
// whole and 14 in four parts, 64 rows of 131072 33 in parts and 32 whole.
int logprob_parts(const int64_t* ntokens, int nranks, size_t vocab) {
  int64_t rows = 0;
  for (int r = 0; r < nranks; ++r) rows += ntokens[r];
  if (rows == 0 || vocab < 65536) return 1;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({gci::kLogprobParts, 256 / rows, static_cast<int64_t>(vocab / 8192)})));
}

}  // namespace

extern "C" size_t gc_token_logprob_scratch_bytes(const int64_t* ntokens, int nranks, size_t vocab, int top) {
  if (logprob_sizes(ntokens, nranks, vocab, top) != GC_OK) return 0;
  const int parts = logprob_parts(ntokens, nranks, vocab);
  uint64_t rows = 0;
  for (int r = 0; r < nranks; ++r) rows += ntokens[r];
  return up256(std::max<uint64_t>(1, parts > 1 ? rows * parts * (16 + 8 * static_cast<uint64_t>(top)) : 0));
}

extern "C" gc_status gc_token_logprob(const void* const* logits, const int32_t* const* targets, const int64_t* ntokens,
                                      int nranks, size_t vocab, size_t stride, float scale, gc_dtype t,
                                      float* const* logprob, float* const* entropy, float* const* lse, int top,
                                      int32_t* const* top_ids, float* const* top_logprob, const float* const* dlogprob,
                                      const float* const* dentropy, void* const* dlogits, void* scratch,
                                      size_t scratch_bytes, hipStream_t stream) {
  GC_TRY(logprob_sizes(ntokens, nranks, vocab, top));
  if (!targets != !logprob || !dlogits != !dlogprob || (dentropy && !dlogits) || (dlogits && !targets))
    return GC_ERR_INVALID_ARG;
  const gci::LogprobCall c{logits, targets, ntokens, nranks, vocab, stride, scale, t, logprob, entropy, lse, top,
                           top_ids, top_logprob, dlogprob, dentropy, dlogits, scratch, stream, logprob_parts(ntokens, nranks, vocab)};
  Buffers b;
  GC_TRY(logprob_check(c, b));
  const auto rows = [&](uint64_t bytes) { return [=](int r) { return static_cast<uint64_t>(ntokens[r]) * bytes; }; };
  for (float* const* p : {logprob, entropy, lse})
    if (p) b.add(any(p), nranks, 4, rows(4), true);
  if (top) {
    b.add(any(top_ids), nranks, 4, rows(4 * static_cast<uint64_t>(top)), true);
    b.add(any(top_logprob), nranks, 4, rows(4 * static_cast<uint64_t>(top)), true);
  }
  const size_t need = gc_token_logprob_scratch_bytes(ntokens, nranks, vocab, top);
  if (scratch_bytes < need) return GC_ERR_INVALID_ARG;
  b.one(scratch, 256, need, true);
  GC_TRY(b.check());
  return gci::launch_token_logprob(c);
}

extern "C" gc_status gc_token_logprob_backward(const void* const* logits, const int32_t* const* targets,
                                               const float* const* lse, const float* const* entropy,
                                               const float* const* dlogprob, const float* const* dentropy,
                                               const int64_t* ntokens, int nranks, size_t vocab, size_t stride,
                                               float scale, gc_dtype t, void* const* dlogits, hipStream_t stream) {
  GC_TRY(logprob_sizes(ntokens, nranks, vocab, 0));
  if (!targets || !dlogprob || !dlogits || (dentropy && !entropy)) return GC_ERR_INVALID_ARG;
  gci::LogprobCall c{};
  c.logits = logits;
  c.targets = targets;
  c.tokens = ntokens;
  c.nranks = nranks;
  c.vocab = vocab;
  c.stride = stride;
  c.scale = scale;
  c.t = t;
  c.lse = const_cast<float* const*>(lse);
  c.entropy = dentropy ? const_cast<float* const*>(entropy) : nullptr;
  c.dlogprob = dlogprob;
  c.dentropy = dentropy;
  c.dlogits = dlogits;
  c.stream = stream;
  Buffers b;
  GC_TRY(logprob_check(c, b));
  const auto per_row = [&](int r) { return static_cast<uint64_t>(ntokens[r]) * 4; };
  b.add(any(lse), nranks, 4, per_row, false);
  if (dentropy) b.add(any(entropy), nranks, 4, per_row, false);
  GC_TRY(b.check());
  return gci::launch_token_logprob_backward(c);
}
