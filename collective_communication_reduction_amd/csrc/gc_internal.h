// Internal interface between the C ABI layer (api.cpp: validation, planning)
// and the kernel launchers (reduce.hip, movement.hip).  Not installed.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "gc.h"

namespace gci {

inline size_t elem_bytes(gc_dtype t) { return t == GC_BF16 ? 2 : 4; }

// Maps a HIP result to a status, remembering a failure for gc_last_hip_error().
gc_status hip_status(hipError_t e);

// Geometry shared by the three reduction-family launches.  The reference index
// space has S elements cut into N chunks [j*c, min(S, (j+1)*c)).
//
//   all_reduce:      in[i]  = rank i's buffer        (element E at in[i] + E)
//                    out[r] = rank r's buffer        (element E at out[r] + E)
//   reduce_scatter:  in[i]  = rank i's full buffer   (element E at in[i] + E)
//                    out[j] = chunk j's destination  (element E at out[j] + E - j*c)
//   all_gather:      in[i]  = shard i                (element E at in[i] + E - i*c)
//                    out[d] = rank d's full buffer   (element E at out[d] + E)
struct ReduceCall {
  const void* const* in;
  void* const* out;
  int nranks;
  uint64_t S;
  uint64_t c;
  gc_dtype in_t;
  gc_dtype out_t;
  bool avg;
  bool ring;
  hipStream_t stream;
  bool wire = false;  // ring whose forwarded partials are rounded to the input type
};

gc_status launch_all_reduce(const ReduceCall& call);

// Two-level reduction over nranks = R * group ranks (rank g * group + i is
// member i of group g).  in[r]: rank r's count elements.  All-reduce: out[r]
// rank r's count elements.  HSDP reduce-scatter: out[r] member i's shard of
// count / group elements.
struct HierCall {
  const void* const* in;
  void* const* out;
  int nranks;
  int group;
  uint64_t count;
  gc_dtype in_t;
  gc_dtype out_t;
  bool avg;
  bool ring;
  hipStream_t stream;
  bool wire = false;  // ring whose forwarded partials are rounded to the input type (both levels)
};

gc_status launch_hier_all_reduce(const HierCall& call);
gc_status launch_hsdp_reduce_scatter(const HierCall& call);
gc_status launch_reduce_scatter(const ReduceCall& call);
gc_status launch_all_gather(const ReduceCall& call);

// Zero-copy bucket all-reduce.  A piece is the part of one tensor that falls
// inside one owner chunk of the bucket's packed index space: elements
// [lo, lo + len) of the tensor in `slot`, folded starting at rank `first`.
struct BucketPiece {
  uint64_t lo;
  uint64_t len;
  uint32_t slot;
  uint32_t first;
};

struct BucketCall {
  void* const* slot_ptrs;  // [nslots * nranks], slot-major: rank r's tensor of slot s at [s * nranks + r]
  int nslots;
  int nranks;
  const BucketPiece* pieces;  // ordered by slot
  int npieces;
  gc_dtype t;
  bool avg;
  double* sumsq;  // device accumulator for the sum of squared results, or nullptr
  hipStream_t stream;
  bool wire = false;  // ring whose forwarded partials are rounded to the input type
};

gc_status launch_bucket_all_reduce(const BucketCall& call);

// Cache policy of a kernel's 16-byte stores.  kStoreNT: the non-temporal hint
// alone.  kStoreDevNT: device scope (sc1) plus the hint: the line is written
// through the XCD's L2 rather than left there dirty.  kStoreDev: device scope
// without the hint, so the line may stay in the MALL for the kernel that reads
// it next.
enum StorePolicy : int { kStoreNT = 0, kStoreDevNT = 1, kStoreDev = 2 };

// One contiguous copy; src == nullptr writes zeros.
struct Segment {
  const void* src;
  void* dst;
  uint64_t bytes;
};

gc_status launch_segment_copy(const Segment* segs, size_t nseg, StorePolicy pol, hipStream_t stream);


// MoE routing plan (see gc_moe_route).  Routes of source s are cut into tiles
// of `tile` routes; counts holds [tiles][nranks * experts_per_rank] int32 and
// roff [nranks][nranks * experts_per_rank] int32 of scratch.
struct MoeRouteCall {
  const int32_t* const* experts;
  int32_t* const* dest;
  const int64_t* routes;  // [nranks] tokens * topk
  int nranks;
  int experts_per_rank;
  int32_t tile;
  int32_t* counts;
  int32_t* roff;
  int64_t* splits;
  hipStream_t stream;
};

// MoE dispatch (src = token rows, dst = receive buffers) or combine
// (src = expert outputs in the receive layout, dst = token rows).
struct MoeMoveCall {
  const void* const* src;
  const int64_t* src_rows;     // rows of each src buffer
  const int32_t* const* dest;  // per source: [tokens * topk] (rank, row) pairs
  const float* const* weights; // combine only
  void* const* dst;
  const int64_t* dst_rows;     // rows of each dst buffer
  const int64_t* tokens;       // [nranks] tokens per source
  int nranks;
  int topk;
  uint64_t row_bytes;
  gc_dtype t;                  // combine only
  hipStream_t stream;
};

// Routes per routing-plan tile while the experts fit it (four wavefronts).
#ifndef GC_MOE_ROUTE_TILE
#define GC_MOE_ROUTE_TILE 1024
#endif
constexpr int32_t kMoeRouteTile = GC_MOE_ROUTE_TILE;

gc_status launch_moe_route(const MoeRouteCall& call);

// Device address of the routing plan's static scratch array on the device that
// runs `stream` (the current device for the null stream), looked up once per
// device; GC_ERR_HIP if the lookup fails.
gc_status moe_route_static_scratch(hipStream_t stream, void** ptr);
gc_status launch_moe_dispatch(const MoeMoveCall& call);
gc_status launch_moe_combine(const MoeMoveCall& call);

// ---- operators of the layer around the experts (norm.hip, mx8.hip, moe_grad.hip, ffn.hip)

// A launch holds fewer than 2^32 work items in a dimension, so a longer grid goes
// in launches of at most 2^31, one after the other on the stream.
// one(first, n) launches workgroups first .. first + n - 1 of `blocks`.
template <class F>
gc_status in_launches(uint64_t blocks, uint32_t threads, F one) {
  const uint64_t most = (uint64_t(1) << 31) / threads;
  for (uint64_t b = 0; b < blocks; b += most) {
    const gc_status st = one(static_cast<uint32_t>(b), static_cast<uint32_t>(blocks - b < most ? blocks - b : most));
    if (st != GC_OK) return st;
  }
  return GC_OK;
}

// A row of n elements is taken in units of `unit`; the last unit of one that is no multiple of it is moved inside the row and
// overlaps the unit before.  A unit may be taken in pieces of `ve` elements, `off` elements into it.
constexpr uint32_t unit_start(uint32_t n, uint32_t unit, uint32_t u) { return n < unit ? 0 : u * unit < n - unit ? u * unit : n - unit; }
// Elements of a piece that lie in the row: all of them but in rows shorter than a unit.
constexpr uint32_t unit_held(uint32_t n, uint32_t unit, uint32_t off, uint32_t ve) {
  return n >= unit ? ve : n <= off ? 0 : n - off < ve ? n - off : ve;
}
// Of these, how many at the piece's front the unit before holds too: whoever adds to the row leaves them to it.
constexpr uint32_t unit_shared(uint32_t n, uint32_t unit, uint32_t u, uint32_t off, uint32_t ve) {
  const uint32_t s = unit_start(n, unit, u) + off, own = u * unit;   // own: the first element that only this unit holds
  return own <= s ? 0 : own - s < ve ? own - s : ve;
}

// Bytes of an 8-bit row of n values: codes, a scale per 32 values, zeros to a multiple of 16.
inline uint64_t mx8_row_bytes(uint64_t n) { return (n + (n + 31) / 32 + 15) / 16 * 16; }

// Token rows of every rank (see gc_rms_norm); res, sum and rstd may be null.
struct NormCall {
  const void* const* x;
  const void* const* res;
  const void* const* w;
  const int64_t* tokens;
  int nranks;
  uint64_t hidden;
  float eps;
  gc_dtype t;
  void* const* sum;
  void* const* y;
  gc_dtype y_t;
  float* const* rstd;
  hipStream_t stream;
};
gc_status launch_rms_norm(const NormCall& call);

struct NormBackwardCall {
  const void* const* dy;
  const void* const* dsum;
  const void* const* sum;
  const void* const* w;
  const float* const* rstd;
  const int64_t* tokens;
  int nranks;
  uint64_t hidden;
  gc_dtype t;
  void* const* dx;
  float* const* dw;
  float* partial;         // [blocks][hidden] partial weight gradients
  int64_t rows_per_block; // consecutive rows of one rank that one block sums
  hipStream_t stream;
};
gc_status launch_rms_norm_backward(const NormBackwardCall& call);

// Rows of n values of type t to 8-bit rows (unpack == false) or back.
struct Mx8Call {
  const void* const* src;
  void* const* dst;
  const int64_t* rows;
  int nranks;
  uint64_t n;
  gc_dtype t;
  bool unpack;
  hipStream_t stream;
};
gc_status launch_mx8(const Mx8Call& call);

struct MoeCombineBackwardCall {
  const void* const* dout;
  const void* const* y;
  const int64_t* y_rows;
  const int32_t* const* dest;
  const float* const* weights;
  const int64_t* tokens;
  int nranks;
  int topk;
  uint64_t hidden;
  gc_dtype t;
  void* const* dy;
  float* const* dweights;
  hipStream_t stream;
};
gc_status launch_moe_combine_backward(const MoeCombineBackwardCall& call);

// Experts (see gc_moe_ffn).  Every per-rank pointer list may be null where a
// direction does not use it.
struct FfnCall {
  const void* const* x;
  gc_dtype x_t;
  const int64_t* rows;
  const int64_t* splits;
  int nranks;
  int experts_per_rank;
  uint64_t hidden;
  uint64_t inter;
  const void* const* w_gate;
  const void* const* w_up;
  const void* const* w_down;
  void* const* saved;        // written by the forward, read by the backward
  gc_dtype saved_t;
  void* const* y;            // forward: output rows; backward: dx rows
  const void* const* dy;     // backward only, as the rest
  void* const* dw_gate;
  void* const* dw_up;
  void* const* dw_down;
  gc_dtype dw_t;
  void* scratch;
  hipStream_t stream;
};

// One expert's block of rows, as the plan kernel leaves it for the products.
struct FfnSeg {
  const char* x;             // first row of each buffer's block
  const char* dy;
  char* saved;
  char* y;
  const char* w_gate;        // this expert's weights and their gradients
  const char* w_up;
  const char* w_down;
  char* dw_gate;
  char* dw_up;
  char* dw_down;
  int64_t row;               // first row in the scratch matrices (all ranks' rows in order)
  int32_t rows;
  int32_t tile0;             // first row tile
};

// Row tiles and the scratch areas of a call, from its sizes alone.
struct FfnGeom {
  int64_t rows = 0;          // of all ranks
  int32_t segs = 0;          // experts of all ranks
  int32_t tile_rows = 0;     // rows per tile of the row products
  bool split = false;        // few rows per expert: h and the gradients of gate and up are kept in two parts
  bool few = false;          // and the serving forward streams the weights instead
  int64_t tiles = 0;         // most row tiles the experts' blocks can make
  uint64_t map = 0, x = 0, h = 0, g = 0, bytes = 0;  // offsets (segment table at 0) and total
};
FfnGeom ffn_geom(const int64_t* rows, int nranks, int experts_per_rank, uint64_t hidden, uint64_t inter, gc_dtype x_t,
                 bool backward);

gc_status launch_moe_ffn(const FfnCall& call);
gc_status launch_moe_ffn_backward(const FfnCall& call);

// ---- the two ends of a training step (embed.hip, dropout.hip, logprob.hip)

// Token lookup (see gc_embedding).
struct EmbeddingCall {
  const void* const* w;
  const int32_t* const* ids;
  const int64_t* tokens;
  int nranks;
  uint64_t vocab;
  uint64_t hidden;
  float scale;
  gc_dtype t;
  void* const* out;
  hipStream_t stream;
};
gc_status launch_embedding(const EmbeddingCall& call);

// Scratch areas of the lookup's gradient, as byte offsets, and its split of the
// tokens: every rank's tokens are sorted in `chunk`-token pieces by two digits
// of the id, the low one of `low_bits` bits.
struct EmbeddingGeom {
  int64_t tokens = 0;   // of all ranks
  int32_t chunk = 0;
  int32_t chunks = 0;   // of all ranks
  int32_t bits = 0;     // of an id
  int32_t low_bits = 0;
  int32_t run = 0;      // sorted tokens that one group of lanes sums
  uint64_t pairs = 0, keys = 0, perm = 0, counts = 0, valid = 0, present = 0, present_row = 0, long_rows = 0, partial = 0, bytes = 0;
};
constexpr int kEmbeddingDigit = 11;   // most bits of a digit
// Floats of a partial row: whole units of either type.
inline uint64_t embedding_pitch(uint64_t hidden) { return (hidden + 7) / 8 * 8; }
EmbeddingGeom embedding_geom(const int64_t* tokens, int nranks, uint64_t vocab, uint64_t hidden);

struct EmbeddingBackwardCall {
  const void* const* dout;
  const int32_t* const* ids;
  const int64_t* tokens;
  int nranks;
  uint64_t vocab;
  uint64_t hidden;
  float scale;
  gc_dtype t;
  void* const* dw;
  gc_dtype dw_t;
  bool accumulate;
  void* scratch;
  EmbeddingGeom geom;
  hipStream_t stream;
};
gc_status launch_embedding_backward(const EmbeddingBackwardCall& call);

// Dropout of every rank's elements (see gc_dropout); res and step may be null.
struct DropoutCall {
  const void* const* x;
  const void* const* res;
  const int64_t* counts;
  int nranks;
  uint32_t drop;        // values whose 16 random bits are below this are dropped
  float scale;          // of the values kept
  uint64_t seed;
  uint64_t offset;
  const uint64_t* step;
  gc_dtype t;
  void* const* y;
  hipStream_t stream;
};
gc_status launch_dropout(const DropoutCall& call);

// Token log probabilities (see gc_token_logprob) and their gradient; which of
// the lists are null says what is asked for.
struct LogprobCall {
  const void* const* logits;
  const int32_t* const* targets;
  const int64_t* tokens;
  int nranks;
  uint64_t vocab;
  uint64_t stride;
  float scale;
  gc_dtype t;
  float* const* logprob;
  float* const* entropy;
  float* const* lse;
  int top;
  int32_t* const* top_ids;
  float* const* top_logprob;
  const float* const* dlogprob;
  const float* const* dentropy;
  void* const* dlogits;
  void* scratch;
  hipStream_t stream;
  int parts = 1;   // of a row where there are few (not with a gradient)
};
constexpr int kLogprobParts = 32;   // at most
gc_status launch_token_logprob(const LogprobCall& call);
gc_status launch_token_logprob_backward(const LogprobCall& call);

}  // namespace gci
