// Argument checks shared by the C ABI files (api*.cpp): buffer extents, spans
// and overlaps on integers, rank and row counts, enums, the buffers of a call.
#pragma once

#include <algorithm>
#include <vector>

#include "gc.h"
#include "gc_internal.h"

#define GC_TRY(expr)                    \
  do {                                  \
    const gc_status _s = (expr);        \
    if (_s != GC_OK) return _s;         \
  } while (0)

namespace gca {

using gci::elem_bytes;

inline bool valid_dtype(gc_dtype t) { return t == GC_INT32 || t == GC_FP32 || t == GC_BF16; }
inline bool valid_op(gc_op op) { return op == GC_SUM || op == GC_AVG; }
inline bool valid_order(gc_order o) { return o == GC_ORDER_RING || o == GC_ORDER_RANK || o == GC_ORDER_RING_WIRE; }

inline uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

// Byte interval [lo, hi) of a buffer.
struct Span {
  uint64_t lo, hi;
  bool empty() const { return hi <= lo; }
};

inline Span span(const void* p, uint64_t bytes) { return Span{addr(p), addr(p) + bytes}; }

// Largest extent of one buffer: 2^40 bytes, beyond any one GPU's memory
// (MI355X: 288 GB of HBM).  With it, and a call's total copy volume bounded by
// kMaxCopyBytes, every tile count the planners derive (2 KiB or more per
// tile) stays below 2^32.
constexpr uint64_t kMaxExtent = uint64_t(1) << 40;
constexpr uint64_t kMaxCopyBytes = uint64_t(1) << 42;

// True if `bytes` bytes at p are a possible buffer: at most kMaxExtent and
// ending inside the 64-bit address space.  Every buffer extent a call derives
// is checked with it before any span is formed, so spans never wrap and the
// addresses handed to the kernels never overflow.
inline bool fits(const void* p, uint64_t bytes) { return bytes <= kMaxExtent && bytes <= UINT64_MAX - addr(p); }

// Address `off` bytes past p, computed on integers (the extent holding it was checked with fits).
inline void* at(const void* p, uint64_t off) { return reinterpret_cast<void*>(addr(p) + off); }

inline bool overlaps(const Span& a, const Span& b) { return !a.empty() && !b.empty() && a.lo < b.hi && b.lo < a.hi; }

// True if any two spans of `w` overlap.
inline bool any_overlap(std::vector<Span> w) {
  std::sort(w.begin(), w.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uint64_t reach = 0;
  bool first = true;
  for (const Span& s : w) {
    if (s.empty()) continue;
    if (!first && s.lo < reach) return true;
    reach = first ? s.hi : std::max(reach, s.hi);
    first = false;
  }
  return false;
}

inline bool mul_overflows(uint64_t a, uint64_t b) { return b != 0 && a > UINT64_MAX / b; }

inline gc_status check_ranks(int nranks) {
  if (nranks < 1) return GC_ERR_INVALID_ARG;
  if (nranks > GC_MAX_RANKS) return GC_ERR_UNSUPPORTED;
  return GC_OK;
}

// n non-null pointers aligned to the element size, each holding `bytes` bytes.
inline gc_status check_ptrs(const void* const* p, int n, size_t es, uint64_t bytes) {
  if (!p) return GC_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!p[i] || addr(p[i]) % es || !fits(p[i], bytes)) return GC_ERR_INVALID_ARG;
  return GC_OK;
}

// Token-row operators: rows of all ranks, and values of one row.
constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr size_t kMaxRow = size_t(1) << 31;

inline bool row_type(gc_dtype t) { return t == GC_BF16 || t == GC_FP32; }

// Buffers of one call: each is checked as it is added (non-null, aligned,
// inside the address space), and at the end no output may overlap another
// buffer.  An input that may coincide with an output is not added where it does.
class Buffers {
 public:
  // n buffers of bytes(i) bytes; empty ones are skipped.
  template <class Bytes>
  void add(const void* const* p, int n, size_t align, Bytes bytes, bool out) {
    if (!p) {
      bad_ = true;
      return;
    }
    for (int i = 0; i < n; ++i) one(p[i], align, bytes(i), out);
  }
  void one(const void* p, size_t align, uint64_t bytes, bool out) {
    if (!bytes) return;
    if (!p || addr(p) % align || !fits(p, bytes)) {
      bad_ = true;
      return;
    }
    (out ? outs_[nout_++] : ins_[nin_++]) = span(p, bytes);
  }
  // No two outputs overlap, and no input overlaps an output.
  gc_status check() {
    if (bad_) return GC_ERR_INVALID_ARG;
    std::sort(outs_, outs_ + nout_, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    for (int k = 1; k < nout_; ++k)
      if (outs_[k].lo < outs_[k - 1].hi) return GC_ERR_INVALID_ARG;
    for (int i = 0; i < nin_; ++i)
      if (hits(ins_[i])) return GC_ERR_INVALID_ARG;
    return GC_OK;
  }

 private:
  // Whether s overlaps an output: the outputs are sorted and disjoint.
  bool hits(const Span& s) const {
    const Span* p = std::lower_bound(outs_, outs_ + nout_, s.lo, [](const Span& o, uint64_t lo) { return o.hi <= lo; });
    return p != outs_ + nout_ && p->lo < s.hi;
  }
  static constexpr int kMost = 8 * GC_MAX_RANKS + 2;
  Span outs_[kMost], ins_[kMost];
  int nout_ = 0, nin_ = 0;
  bool bad_ = false;
};

// Rows per rank, at least 0 and below 2^31 over all ranks.
inline gc_status check_rows(const int64_t* rows, int nranks) {
  GC_TRY(check_ranks(nranks));
  if (!rows) return GC_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int r = 0; r < nranks; ++r) {
    if (rows[r] < 0) return GC_ERR_INVALID_ARG;
    if (rows[r] >= kMaxRows) return GC_ERR_UNSUPPORTED;
    total += rows[r];
  }
  return total >= kMaxRows ? GC_ERR_UNSUPPORTED : GC_OK;
}

// Whether output p[r] is exactly input q[r] (same start; the sizes agree).
inline bool same(const void* const* p, const void* const* q, int r) { return p && q && p[r] == q[r]; }

}  // namespace gca
