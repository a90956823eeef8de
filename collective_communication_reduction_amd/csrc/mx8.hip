// Activation rows to 8-bit rows (e4m3 codes, a power-of-two scale per 32
// values) and back, for gfx950.  Streaming passes: every value is read once and
// written once, so HBM bytes bound them.  A row is shared by a wavefront, or by
// a workgroup where it has more than 8 units per lane of one wavefront; a
// block's maximum is a shuffle over the 32 / VE lanes that hold it.  4 x 8192 bf16
// rows of 11008: 192 us either way, 5.7 TB/s.

#include <type_traits>

#include "rows.h"

namespace {

using namespace gcdev;

constexpr int kMxU = 6;  // units per lane per step, all loaded before the first store (a bf16 row of 11008 at once: 192 us a
                         // pass over 4 x 8192 such rows, against 201 with 4 and 198 with 1 or 2)

template <int P>
struct Mx8Args {
  const char* src[P];
  char* dst[P];
  int64_t rows[P];
  int32_t tile0[P + 1];  // first workgroup of each rank
  uint32_t block0;       // first workgroup of this launch
  uint64_t n;            // values per row
  uint64_t row8;         // bytes per 8-bit row
  int32_t N;
};

template <class In, bool VEC, int LANES, int P>
__global__ void __launch_bounds__(kThreads) mx8_pack_kernel(const Mx8Args<P> a) {
  typedef RowUnit<In, VEC> U;
  typedef typename U::T T;
  constexpr int VE = U::VE;
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int lane = threadIdx.x % LANES;
  const int64_t row = static_cast<int64_t>(block - a.tile0[rank]) * (kThreads / LANES) +
                      threadIdx.x / LANES;
  if (row >= a.rows[rank]) return;
  const uint64_t units = a.n / VE;
  const T* x = reinterpret_cast<const T*>(a.src[rank]) + row * units;
  char* out = a.dst[rank] + row * a.row8;
  for (uint64_t u0 = 0; u0 < units; u0 += kMxU * LANES) {
    T v[kMxU];
#pragma unroll
    for (int j = 0; j < kMxU; ++j) {
      const uint64_t u = u0 + j * LANES + lane;
      v[j] = U::load(x + (u < units ? u : units - 1));
    }
#pragma unroll
    for (int j = 0; j < kMxU; ++j) {
      const uint64_t u = u0 + j * LANES + lane;
      float f[VE];
      U::widen(v[j], f);
      mx8_encode<VE>(out, a.n, u, u < units, f);
    }
  }
  mx8_pad(out, a.n, lane);
}

template <class In, bool VEC, int LANES, int P>
__global__ void __launch_bounds__(kThreads) mx8_unpack_kernel(const Mx8Args<P> a) {
  typedef RowUnit<In, VEC> U;
  typedef typename U::T T;
  constexpr int VE = U::VE;
  typedef typename std::conditional<VE == 8, u32x2, typename std::conditional<VE == 4, uint32_t, uint8_t>::type>::type C;
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int lane = threadIdx.x % LANES;
  const int64_t row = static_cast<int64_t>(block - a.tile0[rank]) * (kThreads / LANES) +
                      threadIdx.x / LANES;
  if (row >= a.rows[rank]) return;
  const uint64_t units = a.n / VE;
  const char* in = a.src[rank] + row * a.row8;
  T* out = reinterpret_cast<T*>(a.dst[rank]) + row * units;
  for (uint64_t u0 = 0; u0 < units; u0 += kMxU * LANES) {
    C c[kMxU];
    uint8_t s[kMxU];
#pragma unroll
    for (int j = 0; j < kMxU; ++j) {
      const uint64_t u = min(u0 + j * LANES + lane, units - 1);
      c[j] = __builtin_nontemporal_load(reinterpret_cast<const C*>(in) + u);
      s[j] = *reinterpret_cast<const uint8_t*>(in + a.n + u / (32 / VE));
    }
#pragma unroll
    for (int j = 0; j < kMxU; ++j) {
      const uint64_t u = u0 + j * LANES + lane;
      if (u >= units) continue;
      const float scale = mx8_scale(s[j]);
      float v[VE];
      if constexpr (VE == 1) {
        v[0] = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[j]), false)[0] * scale;
      } else {
#pragma unroll
        for (int q = 0; q < VE / 4; ++q) {
          float f[4];
          uint32_t w;
          if constexpr (VE == 8) w = c[j][q];
          else w = c[j];
          mx8_values(w, scale, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * q + e] = f[e];
        }
      }
      U::store(out + u, U::narrow(v));
    }
  }
}

template <class In, bool VEC, int P>
gc_status mx8_impl(const gci::Mx8Call& c, Mx8Args<P>& a) {
  const bool wave = c.n / RowUnit<In, VEC>::VE <= 8 * kWave;
  const int64_t per = wave ? kThreads / kWave : 1;
  int32_t run = 0;
  for (int s = 0; s < c.nranks; ++s) {
    a.tile0[s] = run;
    run += static_cast<int32_t>((c.rows[s] + per - 1) / per);
  }
  for (int s = c.nranks; s <= P; ++s) a.tile0[s] = run;
  void* params[] = {&a};
  const void* k;
  if (c.unpack) k = wave ? reinterpret_cast<const void*>(mx8_unpack_kernel<In, VEC, kWave, P>)
                         : reinterpret_cast<const void*>(mx8_unpack_kernel<In, VEC, kThreads, P>);
  else k = wave ? reinterpret_cast<const void*>(mx8_pack_kernel<In, VEC, kWave, P>)
                : reinterpret_cast<const void*>(mx8_pack_kernel<In, VEC, kThreads, P>);
  return gci::in_launches(run, kThreads, [&](uint32_t first, uint32_t blocks) {
    a.block0 = first;
    return gci::hip_status(hipLaunchKernel(k, dim3(blocks), dim3(kThreads), params, 0, c.stream));
  });
}

template <class In, int P>
gc_status mx8_typed(const gci::Mx8Call& c) {
  Mx8Args<P> a{};
  uint64_t m = c.n * In::ES;
  for (int s = 0; s < c.nranks; ++s) {
    a.src[s] = static_cast<const char*>(c.src[s]);
    a.dst[s] = static_cast<char*>(c.dst[s]);
    a.rows[s] = c.rows[s];
    if (c.rows[s]) m |= reinterpret_cast<uint64_t>(c.unpack ? c.dst[s] : c.src[s]);
  }
  a.n = c.n;
  a.row8 = gci::mx8_row_bytes(c.n);
  a.N = c.nranks;
  return (m & 15) == 0 ? mx8_impl<In, true, P>(c, a) : mx8_impl<In, false, P>(c, a);
}

}  // namespace

namespace gci {

gc_status launch_mx8(const Mx8Call& c) {
  if (c.t == GC_BF16) return c.nranks <= 8 ? mx8_typed<InBf16, 8>(c) : mx8_typed<InBf16, 64>(c);
  return c.nranks <= 8 ? mx8_typed<InF32, 8>(c) : mx8_typed<InF32, 64>(c);
}

}  // namespace gci
