// Host-only stand-ins for the launchers of the layer operators, for the
// sanitizer build of api_layer.cpp: every byte range a launch would touch must
// lie inside a buffer the harness declared with the extent the contract gives.
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
}  // namespace

void reset() { g_bufs.clear(); }
void declare(const void* p, uint64_t bytes) {
  if (p && bytes) g_bufs.push_back(Buf{addr(p), addr(p) + bytes});
}
long launches() { return g_launches; }
long violations() { return g_bad; }

}  // namespace stub

namespace gci {

using stub::need;

gc_status launch_mx8(const Mx8Call& c) {
  const uint64_t dense = c.n * elem_bytes(c.t), packed = mx8_row_bytes(c.n);
  for (int r = 0; r < c.nranks; ++r) {
    need(c.src[r], c.rows[r] * (c.unpack ? packed : dense), "8-bit rows source");
    need(c.dst[r], c.rows[r] * (c.unpack ? dense : packed), "8-bit rows destination");
  }
  ++stub::g_launches;
  return GC_OK;
}

gc_status launch_rms_norm(const NormCall& c) {
  const uint64_t row = c.hidden * elem_bytes(c.t);
  for (int r = 0; r < c.nranks; ++r) {
    const uint64_t n = c.tokens[r];
    need(c.x[r], n * row, "norm x");
    if (c.res) need(c.res[r], n * row, "norm residual");
    if (n) need(c.w[r], row, "norm weight");
    if (c.sum) need(c.sum[r], n * row, "norm sum");
    need(c.y[r], n * (c.y_t == GC_MX8 ? mx8_row_bytes(c.hidden) : row), "norm y");
    if (c.rstd) need(c.rstd[r], n * 4, "norm rstd");
  }
  ++stub::g_launches;
  return GC_OK;
}

gc_status launch_rms_norm_backward(const NormBackwardCall& c) {
  const uint64_t row = c.hidden * elem_bytes(c.t);
  uint64_t blocks = 0;
  for (int r = 0; r < c.nranks; ++r) {
    const uint64_t n = c.tokens[r];
    need(c.dy[r], n * row, "norm dy");
    if (c.dsum) need(c.dsum[r], n * row, "norm dsum");
    need(c.sum[r], n * row, "norm sum");
    if (n) need(c.w[r], row, "norm weight");
    need(c.rstd[r], n * 4, "norm rstd");
    need(c.dx[r], n * row, "norm dx");
    need(c.dw[r], c.hidden * 4, "norm dweight");
    blocks += (n + c.rows_per_block - 1) / c.rows_per_block;
  }
  need(c.partial, blocks * c.hidden * 4, "norm partial sums");
  ++stub::g_launches;
  return GC_OK;
}

gc_status launch_moe_combine_backward(const MoeCombineBackwardCall& c) {
  const uint64_t row = c.hidden * elem_bytes(c.t);
  for (int r = 0; r < c.nranks; ++r) {
    const uint64_t routes = static_cast<uint64_t>(c.tokens[r]) * c.topk;
    need(c.dout[r], c.tokens[r] * row, "combine dout");
    need(c.y[r], c.y_rows[r] * row, "combine expert rows");
    need(c.dy[r], c.y_rows[r] * row, "combine gradient rows");
    need(c.dest[r], routes * 8, "combine dest");
    need(c.weights[r], routes * 4, "combine weights");
    need(c.dweights[r], routes * 4, "combine weight gradients");
  }
  ++stub::g_launches;
  return GC_OK;
}

static gc_status ffn_like(const FfnCall& c, bool backward) {
  const FfnGeom g = ffn_geom(c.rows, c.nranks, c.experts_per_rank, c.hidden, c.inter, c.x_t, backward);
  const uint64_t w = static_cast<uint64_t>(c.experts_per_rank) * c.hidden * c.inter;
  const uint64_t saved = c.saved_t == GC_MX8 ? mx8_row_bytes(2 * c.inter) : c.inter * 4;
  int64_t tiles = 0;
  for (int r = 0; r < c.nranks; ++r) {
    const uint64_t n = c.rows[r];
    need(c.x[r], n * (c.x_t == GC_MX8 ? mx8_row_bytes(c.hidden) : c.hidden * 2), "experts x");
    need(c.w_gate[r], w * 2, "experts gate");
    need(c.w_up[r], w * 2, "experts up");
    need(c.w_down[r], w * 2, "experts down");
    if (c.saved) need(c.saved[r], n * saved, "experts checkpoint");
    need(c.y[r], n * c.hidden * 2, "experts rows out");
    if (backward) {
      const uint64_t e = c.dw_t == GC_FP32 ? 4 : 2;
      need(c.dy[r], n * c.hidden * 2, "experts dy");
      need(c.dw_gate[r], w * e, "experts gate gradient");
      need(c.dw_up[r], w * e, "experts up gradient");
      need(c.dw_down[r], w * e, "experts down gradient");
    }
    // the most tiles E blocks can cut n rows into
    const int64_t blocks = std::min<int64_t>(c.experts_per_rank, n);
    tiles += blocks ? blocks + (static_cast<int64_t>(n) - blocks) / g.tile_rows : 0;
  }
  if (tiles > g.tiles) ++stub::g_bad;
  need(c.splits, static_cast<uint64_t>(c.nranks) * c.nranks * c.experts_per_rank * 8, "experts splits");
  need(c.scratch, g.bytes, "experts scratch");
  ++stub::g_launches;
  return GC_OK;
}
gc_status launch_moe_ffn(const FfnCall& c) { return ffn_like(c, false); }
gc_status launch_moe_ffn_backward(const FfnCall& c) { return ffn_like(c, true); }

}  // namespace gci
