// Argument checks shared by the C ABI files (api.cpp, api_layer.cpp): buffer
// extents, spans and overlaps on integers, rank counts and enums.
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

}  // namespace gca
