// Dropout with the residual's addition, from a counter-based generator, for gfx950.
//
//   y = residual + keep * x / (1 - p)
//
// keep of element i depends on (seed, offset + step, rank, i) alone: words of
// Philox4x32-10 (J. Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011), so no mask is ever stored and the gradient's call makes the same one.
// One 128-bit block of the generator serves eight elements, 16 bits each: with 32
// bits each the generator's 20 quarter-rate products per block, not HBM, would
// bound bf16 rows.

#include <type_traits>

#include "units.h"

namespace {

using namespace gcdev;

constexpr int kPer = 8;   // elements of one generator block

template <int P>
struct DropoutArgs {
  const char* x[P];
  const char* res[P];
  char* y[P];
  int64_t n[P];
  int32_t tile0[P + 1];
  uint32_t block0;
  int32_t N;
  uint32_t key0, key1;
  uint64_t offset;
  const uint64_t* step;
  uint32_t drop;
  float scale;
  bool through;   // every y starts on a line
};

__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c[0], b = static_cast<uint64_t>(0xCD9E8D57u) * c[2];
    const uint32_t c1 = c[1], c3 = c[3];
    c[0] = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c[1] = static_cast<uint32_t>(b);
    c[2] = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c[3] = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// A lane takes one unit, a whole generator block of bf16 elements or half of one of
// fp32: with both halves in one lane each of its stores would leave every other 16
// bytes to the next store (2.4 TB/s instead of 6).  A workgroup takes kThreads units.
// HBM bounds it: 8 x 16384 x 4096 bf16 with residual 500 us, 6.4 TB/s, near the library's
// copies; 4 ranks of as many fp32 values 506 us.
template <class In, bool RES, int P>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutArgs<P> a) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE, PER = kPer / VE;   // units per generator block
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const uint64_t first = static_cast<uint64_t>(block - a.tile0[rank]) * (kThreads * VE);   // the workgroup's elements
  const uint32_t n = static_cast<uint32_t>(min<uint64_t>(kThreads * VE, a.n[rank] - first));
  if (threadIdx.x * VE >= n) return;
  const uint32_t here = min(n - threadIdx.x * VE, static_cast<uint32_t>(VE));   // elements of the unit
  const uint64_t off = (first + threadIdx.x * VE) * In::ES;
  const u32x4 x = U::load(a.x[rank] + off, here, 0);
  u32x4 r;
  if (RES) r = U::load(a.res[rank] + off, here, 0);
  const uint64_t u = first / VE + threadIdx.x;
  const uint64_t at = a.offset + (a.step ? *a.step : 0), b = u / PER;
  uint32_t c[4] = {static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32) | static_cast<uint32_t>(rank) << 8,
                   static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32)};
  philox(c, a.key0, a.key1);
  if (PER == 2 && u % 2) {
    c[0] = c[2];
    c[1] = c[3];
  }
  float v[VE], s[VE];
  U::widen(x, v);
  if (RES) U::widen(r, s);
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const uint32_t bits = e % 2 ? c[e / 2] >> 16 : c[e / 2] & 0xFFFFu;
    const float k = bits >= a.drop ? v[e] * a.scale : 0.0f;  // a dropped value counts as 0, whatever it is
    v[e] = RES ? s[e] + k : k;
  }
  U::store(a.y[rank] + off, here, 0, U::narrow(v), a.through);
}

template <class In, int P>
gc_status dropout_typed(const gci::DropoutCall& c) {
  DropoutArgs<P> a{};
  for (int s = 0; s < c.nranks; ++s) {
    a.x[s] = static_cast<const char*>(c.x[s]);
    if (c.res) a.res[s] = static_cast<const char*>(c.res[s]);
    a.y[s] = static_cast<char*>(c.y[s]);
    a.n[s] = c.counts[s];
  }
  if (!fill_blocks<P>(a.tile0, c.counts, c.nranks, kThreads * In::VE)) return GC_ERR_UNSUPPORTED;
  uint64_t m = 0;
  for (int s = 0; s < c.nranks; ++s) m |= c.counts[s] ? reinterpret_cast<uint64_t>(c.y[s]) : 0;
  a.through = m % kLine == 0;
  a.N = c.nranks;
  a.key0 = static_cast<uint32_t>(c.seed);
  a.key1 = static_cast<uint32_t>(c.seed >> 32);
  a.offset = c.offset;
  a.step = c.step;
  a.drop = c.drop;
  a.scale = c.scale;
  const int32_t g = a.tile0[c.nranks];
  return c.res ? launch_blocks(dropout_kernel<In, true, P>, a, g, kThreads, c.stream)
               : launch_blocks(dropout_kernel<In, false, P>, a, g, kThreads, c.stream);
}

}  // namespace

namespace gci {

gc_status launch_dropout(const DropoutCall& c) {
  if (c.t == GC_BF16) return c.nranks <= 8 ? dropout_typed<InBf16, 8>(c) : dropout_typed<InBf16, 64>(c);
  return c.nranks <= 8 ? dropout_typed<InF32, 8>(c) : dropout_typed<InF32, 64>(c);
}

}  // namespace gci
