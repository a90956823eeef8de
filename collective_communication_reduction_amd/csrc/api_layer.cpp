// C ABI of the layer around the experts: residual RMS norm, 8-bit rows, the
// gradient of the MoE combine and the experts' gated feed-forward block.
// Argument validation and aliasing rules, then the launches.  Every check runs
// before anything is enqueued, and nothing here allocates.

#include "api_checks.h"

namespace {

using namespace gca;

constexpr int kMaxTopk = 8;
constexpr int kMaxExperts = 8192;
constexpr size_t kMaxDim = size_t(1) << 20;   // hidden and inter of the experts

}  // namespace

// ------------------------------------------------------------- 8-bit rows

extern "C" size_t gc_mx8_row_bytes(size_t n) {
  return n == 0 || n > kMaxRow ? 0 : static_cast<size_t>(gci::mx8_row_bytes(n));
}

namespace {

gc_status mx8_call(const void* const* src, const int64_t* rows, int nranks, size_t n, gc_dtype t, void* const* dst,
                   bool unpack, hipStream_t stream) {
  GC_TRY(check_rows(rows, nranks));
  if (n == 0) return GC_ERR_INVALID_ARG;
  if (n > kMaxRow) return GC_ERR_UNSUPPORTED;
  if (t != GC_MX8 && !valid_dtype(t)) return GC_ERR_INVALID_ARG;
  if (!row_type(t)) return GC_ERR_UNSUPPORTED;
  const size_t es = elem_bytes(t);
  const uint64_t dense = n * es, packed = gci::mx8_row_bytes(n);
  Buffers b;
  b.add(src, nranks, unpack ? 16 : es, [&](int r) { return rows[r] * (unpack ? packed : dense); }, false);
  b.add(const_cast<const void* const*>(dst), nranks, unpack ? es : 16,
        [&](int r) { return rows[r] * (unpack ? dense : packed); }, true);
  GC_TRY(b.check());
  gci::Mx8Call call{src, dst, rows, nranks, n, t, unpack, stream};
  return gci::launch_mx8(call);
}

}  // namespace

extern "C" gc_status gc_mx8_pack(const void* const* x, const int64_t* rows, int nranks, size_t n, gc_dtype t,
                                 void* const* packed, hipStream_t stream) {
  return mx8_call(x, rows, nranks, n, t, packed, false, stream);
}

extern "C" gc_status gc_mx8_unpack(const void* const* packed, const int64_t* rows, int nranks, size_t n, gc_dtype t,
                                   void* const* out, hipStream_t stream) {
  return mx8_call(packed, rows, nranks, n, t, out, true, stream);
}

// ------------------------------------------------------------- norm

extern "C" gc_status gc_rms_norm(const void* const* x, const void* const* residual, const void* const* weight,
                                 const int64_t* ntokens, int nranks, size_t hidden, float eps, gc_dtype t,
                                 void* const* sum_out, void* const* y, gc_dtype y_t, float* const* rstd,
                                 hipStream_t stream) {
  GC_TRY(check_rows(ntokens, nranks));
  if (hidden == 0 || !(eps >= 0.0f) || eps > 3.4e38f) return GC_ERR_INVALID_ARG;
  if (hidden > kMaxRow) return GC_ERR_UNSUPPORTED;
  if ((t != GC_MX8 && !valid_dtype(t)) || (y_t != GC_MX8 && !valid_dtype(y_t))) return GC_ERR_INVALID_ARG;
  if (!row_type(t) || (y_t != t && y_t != GC_MX8)) return GC_ERR_UNSUPPORTED;
  const size_t es = elem_bytes(t);
  const uint64_t row = hidden * es, y_row = y_t == GC_MX8 ? gci::mx8_row_bytes(hidden) : row;
  const auto bytes = [&](int r) { return static_cast<uint64_t>(ntokens[r]) * row; };
  Buffers b;
  // x and residual: left out of the overlap check where sum_out is that very buffer
  b.add(x, nranks, es, [&](int r) { return same(sum_out, x, r) ? 0 : bytes(r); }, false);
  if (residual) b.add(residual, nranks, es, [&](int r) { return same(sum_out, residual, r) ? 0 : bytes(r); }, false);
  b.add(weight, nranks, es, [&](int r) { return ntokens[r] ? row : 0; }, false);
  if (sum_out) b.add(const_cast<const void* const*>(sum_out), nranks, es, bytes, true);
  b.add(const_cast<const void* const*>(y), nranks, y_t == GC_MX8 ? 16 : es,
        [&](int r) { return static_cast<uint64_t>(ntokens[r]) * y_row; }, true);
  if (rstd)
    b.add(reinterpret_cast<const void* const*>(rstd), nranks, 4,
          [&](int r) { return static_cast<uint64_t>(ntokens[r]) * 4; }, true);
  GC_TRY(b.check());
  gci::NormCall call{x, residual, weight, ntokens, nranks, hidden, eps, t, sum_out, y, y_t, rstd, stream};
  return gci::launch_rms_norm(call);
}

namespace {

// Consecutive rows of one rank per block of the backward: about a thousand
// blocks over all ranks (four per CU), at least four rows each, so that the
// partial weight gradients stay a small part of the rows' own bytes.
int64_t norm_rows_per_block(const int64_t* ntokens, int nranks) {
  int64_t total = 0;
  for (int r = 0; r < nranks; ++r) total += ntokens[r];
  return std::max<int64_t>(4, (total + 1023) / 1024);
}

uint64_t norm_partial_bytes(const int64_t* ntokens, int nranks, size_t hidden) {
  const int64_t per = norm_rows_per_block(ntokens, nranks);
  uint64_t blocks = 0;
  for (int r = 0; r < nranks; ++r) blocks += static_cast<uint64_t>((ntokens[r] + per - 1) / per);
  return std::max<uint64_t>(256, (blocks * hidden * 4 + 255) / 256 * 256);
}

}  // namespace

extern "C" size_t gc_rms_norm_backward_scratch_bytes(const int64_t* ntokens, int nranks, size_t hidden) {
  if (check_rows(ntokens, nranks) != GC_OK || hidden == 0 || hidden > kMaxRow) return 0;
  return norm_partial_bytes(ntokens, nranks, hidden);
}

extern "C" gc_status gc_rms_norm_backward(const void* const* dy, const void* const* dsum, const void* const* sum,
                                          const void* const* weight, const float* const* rstd, const int64_t* ntokens,
                                          int nranks, size_t hidden, gc_dtype t, void* const* dx,
                                          float* const* dweight, void* scratch, size_t scratch_bytes,
                                          hipStream_t stream) {
  GC_TRY(check_rows(ntokens, nranks));
  if (hidden == 0 || (t != GC_MX8 && !valid_dtype(t))) return GC_ERR_INVALID_ARG;
  if (hidden > kMaxRow || !row_type(t)) return GC_ERR_UNSUPPORTED;
  const uint64_t need = norm_partial_bytes(ntokens, nranks, hidden);
  if (scratch_bytes < need) return GC_ERR_INVALID_ARG;
  const size_t es = elem_bytes(t);
  const uint64_t row = hidden * es;
  const auto bytes = [&](int r) { return static_cast<uint64_t>(ntokens[r]) * row; };
  Buffers b;
  b.add(dy, nranks, es, [&](int r) { return same(dx, dy, r) ? 0 : bytes(r); }, false);
  if (dsum) b.add(dsum, nranks, es, [&](int r) { return same(dx, dsum, r) ? 0 : bytes(r); }, false);
  b.add(sum, nranks, es, bytes, false);
  b.add(weight, nranks, es, [&](int r) { return ntokens[r] ? row : 0; }, false);
  b.add(reinterpret_cast<const void* const*>(rstd), nranks, 4,
        [&](int r) { return static_cast<uint64_t>(ntokens[r]) * 4; }, false);
  b.add(const_cast<const void* const*>(dx), nranks, es, bytes, true);
  b.add(reinterpret_cast<const void* const*>(dweight), nranks, 4, [&](int) { return hidden * 4; }, true);
  b.one(scratch, 256, need, true);
  GC_TRY(b.check());
  gci::NormBackwardCall call{dy, dsum, sum, weight, rstd, ntokens, nranks, hidden, t, dx, dweight,
                             static_cast<float*>(scratch), norm_rows_per_block(ntokens, nranks), stream};
  return gci::launch_rms_norm_backward(call);
}

// ------------------------------------------------------------- combine gradient

extern "C" gc_status gc_moe_combine_backward(const void* const* dout, const void* const* expert_out,
                                             const int64_t* expert_rows, const int32_t* const* dest,
                                             const float* const* weights, const int64_t* ntokens, int nranks,
                                             int topk, size_t hidden, gc_dtype t, void* const* dexpert,
                                             float* const* dweights, hipStream_t stream) {
  GC_TRY(check_rows(ntokens, nranks));
  GC_TRY(check_rows(expert_rows, nranks));
  if (topk < 1 || hidden == 0 || (t != GC_MX8 && !valid_dtype(t))) return GC_ERR_INVALID_ARG;
  if (topk > kMaxTopk || hidden > kMaxRow || !row_type(t)) return GC_ERR_UNSUPPORTED;
  int64_t routes = 0;
  for (int r = 0; r < nranks; ++r) routes += ntokens[r] * topk;
  if (routes >= kMaxRows) return GC_ERR_UNSUPPORTED;
  const size_t es = elem_bytes(t);
  const uint64_t row = hidden * es;
  const auto token_rows = [&](int r) { return static_cast<uint64_t>(ntokens[r]) * row; };
  const auto expert_bytes = [&](int r) { return static_cast<uint64_t>(expert_rows[r]) * row; };
  const auto per_route = [&](uint64_t b) {
    return [=](int r) { return static_cast<uint64_t>(ntokens[r]) * topk * b; };
  };
  Buffers b;
  b.add(dout, nranks, es, token_rows, false);
  b.add(expert_out, nranks, es, expert_bytes, false);
  b.add(reinterpret_cast<const void* const*>(dest), nranks, 8, per_route(8), false);
  b.add(reinterpret_cast<const void* const*>(weights), nranks, 4, per_route(4), false);
  b.add(const_cast<const void* const*>(dexpert), nranks, es, expert_bytes, true);
  b.add(reinterpret_cast<const void* const*>(dweights), nranks, 4, per_route(4), true);
  GC_TRY(b.check());
  gci::MoeCombineBackwardCall call{dout, expert_out, expert_rows, dest, weights, ntokens, nranks, topk, hidden, t,
                                   dexpert, dweights, stream};
  return gci::launch_moe_combine_backward(call);
}

// ------------------------------------------------------------- experts

namespace {
uint64_t up64(uint64_t x) { return (x + 63) & ~uint64_t(63); }
uint64_t up256(uint64_t x) { return (x + 255) & ~uint64_t(255); }
}  // namespace

// Row tiles follow the mean block: a tile's rows past its block are computed
// and dropped, so few rows per expert take lower tiles.  A serving forward of a
// handful of rows streams the weights instead.  It reads an expert's weights once
// per 16 rows of that expert (down: 8), and the host does not know which expert gets
// them, so the rule bounds the rows of all of them: us streamed / in tiles, for rows
// spread evenly, as 1 / k over the experts, all on one:
//     16 experts of 2048 x 1024, 16 rows     48 / 58    45 / 47    47 / 43
//                                32          52 / 74    51 / 65    90 / 44
//                                64          61 / 75    77 / 68   175 / 44
//      8 experts of 4096 x 11008, 16        376 / 502  372 / 487  123 / 295
//                                32         489 / 554  486 / 525  225 / 312
//     64 experts of 4096 x 1024, 32         156 / 164  116 / 138   99 / 64
//                                64         225 / 235  170 / 175  189 / 66
//                               256         338 / 317  395 / 266  721 / 83
// Each of its workgroups also adds up its rank's table up to its expert, and every
// expert has workgroups: 256 of 2048 x 1024 with 8 rows take 77 / 56, 74 / 45, 59 / 44.
constexpr int kFewRows = 32, kFewSegs = 64;

// With few rows per expert, or few in all, h and the gradients of gate and up are
// kept in two parts: a single bf16 rounding of them adds about as much to the
// results' 2-norm error as the results' own rounding (sqrt 2 together), and with few
// rows its share of single results spreads to twice that.  It costs a backward of 64
// rows over 16 experts of 2048 x 1024 160 us against 147 (three routings), a forward
// of 40 rows in tiles over 8 of 4096 x 11008 509 against 501.
gci::FfnGeom gci::ffn_geom(const int64_t* rows, int nranks, int E, uint64_t hidden, uint64_t inter, gc_dtype x_t, bool backward) {
  gci::FfnGeom g;
  for (int d = 0; d < nranks; ++d) g.rows += rows[d];
  g.segs = nranks * E;
  const int64_t avg = g.rows / g.segs;
  g.split = avg < 8 || g.rows < 64;
  g.tile_rows = avg >= 192 ? 256 : avg >= 96 ? 128 : g.split ? 32 : 64;
  g.few = avg < 8 && g.rows <= kFewRows && g.segs <= kFewSegs;
  const uint64_t part = g.split ? 2 * up64(inter) : inter;  // values of h per row
  for (int d = 0; d < nranks; ++d) g.tiles += rows[d] / g.tile_rows + std::min<int64_t>(E, rows[d]);
  g.map = up256(static_cast<uint64_t>(g.segs) * sizeof(gci::FfnSeg));
  g.x = g.map + up256(static_cast<uint64_t>(g.tiles) * 4);
  g.h = g.x + (x_t == GC_MX8 ? up256(static_cast<uint64_t>(g.rows) * hidden * 2) : 0);
  g.g = g.h + up256(static_cast<uint64_t>(g.rows) * part * 2);
  g.bytes = g.g + (backward ? up256(static_cast<uint64_t>(g.rows) * part * 4) : 0);
  return g;
}

namespace {

gc_status ffn_sizes(const int64_t* rows, int nranks, int E, size_t hidden, size_t inter, gc_dtype x_t) {
  GC_TRY(check_rows(rows, nranks));
  if (E < 1 || hidden == 0 || inter == 0 || (x_t != GC_MX8 && !valid_dtype(x_t))) return GC_ERR_INVALID_ARG;
  if (static_cast<int64_t>(nranks) * E > kMaxExperts || hidden > kMaxDim || inter > kMaxDim || hidden % 8 || inter % 8 ||
      (x_t != GC_MX8 && x_t != GC_BF16))
    return GC_ERR_UNSUPPORTED;
  return GC_OK;
}

// What both directions check; the buffers that one of them adds are in b already.
gc_status ffn_check(const gci::FfnCall& c, size_t scratch_bytes, bool backward, Buffers& b) {
  if (c.saved) {
    if (c.saved_t != GC_MX8 && !valid_dtype(c.saved_t)) return GC_ERR_INVALID_ARG;
    if (c.saved_t != GC_MX8 && c.saved_t != GC_BF16) return GC_ERR_UNSUPPORTED;
    if (c.saved_t == GC_MX8 && c.inter % 32) return GC_ERR_UNSUPPORTED;
  }
  const int N = c.nranks;
  const uint64_t x_row = c.x_t == GC_MX8 ? gci::mx8_row_bytes(c.hidden) : c.hidden * 2;
  const uint64_t saved_row = c.saved_t == GC_MX8 ? gci::mx8_row_bytes(2 * c.inter) : c.inter * 4;
  const uint64_t w = static_cast<uint64_t>(c.experts_per_rank) * c.hidden * c.inter * 2;
  const auto rows_of = [&](uint64_t row) { return [&c, row](int r) { return static_cast<uint64_t>(c.rows[r]) * row; }; };
  const auto weights = [&](int) { return w; };
  b.add(c.x, N, 16, rows_of(x_row), false);
  b.one(c.splits, 8, static_cast<uint64_t>(N) * N * c.experts_per_rank * 8, false);
  b.add(c.w_gate, N, 16, weights, false);
  b.add(c.w_up, N, 16, weights, false);
  b.add(c.w_down, N, 16, weights, false);
  if (c.saved) b.add(const_cast<const void* const*>(c.saved), N, 16, rows_of(saved_row), !backward);
  b.add(const_cast<const void* const*>(c.y), N, 16, rows_of(c.hidden * 2), true);
  const gci::FfnGeom g = gci::ffn_geom(c.rows, N, c.experts_per_rank, c.hidden, c.inter, c.x_t, backward);
  if (scratch_bytes < g.bytes) return GC_ERR_INVALID_ARG;
  b.one(c.scratch, 256, g.bytes, true);
  // Tiles of each product: 32-bit numbers.  Buffers that could make 2^31 of them are past kMaxExtent in any case.
  const auto tiles = [](uint64_t m, uint64_t n, uint64_t by) { return m * ((n + by - 1) / by); };
  uint64_t most = std::max(tiles(g.tiles, c.inter, 128), tiles(g.tiles, c.hidden, 256));
  if (backward) most = std::max(most, tiles(tiles(g.segs, 2 * up64(c.inter), 256), c.hidden, 256));
  if (most >= (uint64_t(1) << 31)) return GC_ERR_UNSUPPORTED;
  return b.check();
}

}  // namespace

extern "C" size_t gc_moe_ffn_scratch_bytes(const int64_t* rows, int nranks, int experts_per_rank, size_t hidden,
                                           size_t inter, gc_dtype x_t, int backward) {
  if (ffn_sizes(rows, nranks, experts_per_rank, hidden, inter, x_t) != GC_OK) return 0;
  return gci::ffn_geom(rows, nranks, experts_per_rank, hidden, inter, x_t, backward != 0).bytes;
}

extern "C" gc_status gc_moe_ffn(const void* const* x, gc_dtype x_t, const int64_t* rows, const int64_t* splits,
                                int nranks, int experts_per_rank, size_t hidden, size_t inter,
                                const void* const* w_gate, const void* const* w_up, const void* const* w_down,
                                void* const* saved, gc_dtype saved_t, void* const* y, void* scratch,
                                size_t scratch_bytes, hipStream_t stream) {
  GC_TRY(ffn_sizes(rows, nranks, experts_per_rank, hidden, inter, x_t));
  gci::FfnCall c{};
  c.x = x;
  c.x_t = x_t;
  c.rows = rows;
  c.splits = splits;
  c.nranks = nranks;
  c.experts_per_rank = experts_per_rank;
  c.hidden = hidden;
  c.inter = inter;
  c.w_gate = w_gate;
  c.w_up = w_up;
  c.w_down = w_down;
  c.saved = saved;
  c.saved_t = saved_t;
  c.y = y;
  c.scratch = scratch;
  c.stream = stream;
  Buffers b;
  GC_TRY(ffn_check(c, scratch_bytes, false, b));
  return gci::launch_moe_ffn(c);
}

extern "C" gc_status gc_moe_ffn_backward(const void* const* dy, const void* const* x, gc_dtype x_t,
                                         const void* const* saved, gc_dtype saved_t, const int64_t* rows,
                                         const int64_t* splits, int nranks, int experts_per_rank, size_t hidden,
                                         size_t inter, const void* const* w_gate, const void* const* w_up,
                                         const void* const* w_down, void* const* dx, void* const* dw_gate,
                                         void* const* dw_up, void* const* dw_down, gc_dtype dw_t, void* scratch,
                                         size_t scratch_bytes, hipStream_t stream) {
  GC_TRY(ffn_sizes(rows, nranks, experts_per_rank, hidden, inter, x_t));
  if (!saved || (dw_t != GC_MX8 && !valid_dtype(dw_t))) return GC_ERR_INVALID_ARG;
  if (!row_type(dw_t)) return GC_ERR_UNSUPPORTED;
  gci::FfnCall c{};
  c.x = x;
  c.x_t = x_t;
  c.rows = rows;
  c.splits = splits;
  c.nranks = nranks;
  c.experts_per_rank = experts_per_rank;
  c.hidden = hidden;
  c.inter = inter;
  c.w_gate = w_gate;
  c.w_up = w_up;
  c.w_down = w_down;
  c.saved = const_cast<void* const*>(saved);
  c.saved_t = saved_t;
  c.y = dx;
  c.dy = dy;
  c.dw_gate = dw_gate;
  c.dw_up = dw_up;
  c.dw_down = dw_down;
  c.dw_t = dw_t;
  c.scratch = scratch;
  c.stream = stream;
  Buffers b;
  const uint64_t dw = static_cast<uint64_t>(experts_per_rank) * hidden * inter * elem_bytes(dw_t);
  b.add(dy, nranks, 16, [&](int r) { return static_cast<uint64_t>(rows[r]) * hidden * 2; }, false);
  for (void* const* p : {dw_gate, dw_up, dw_down})
    b.add(const_cast<const void* const*>(p), nranks, 16, [&](int) { return dw; }, true);
  GC_TRY(ffn_check(c, scratch_bytes, true, b));
  return gci::launch_moe_ffn_backward(c);
}
