// Device helpers of the row operators (norm, 8-bit rows, combine gradient):
// units of a row (a 16-byte vector, or one element where rows are not 16-byte
// aligned), sums over a wavefront or workgroup, and the 8-bit row format.
#pragma once

#include "fold.h"
#include "gc_internal.h"

namespace gcdev {

constexpr int kWave = 64;

// Rank of tile b, first[s] the first tile of rank s: at most N - 1 steps on uniform values.
template <int P>
__device__ __forceinline__ int rank_of(const int32_t (&first)[P + 1], int N, int32_t b) {
  int s = 0;
  while (s + 1 < N && first[s + 1] <= b) ++s;
  return s;
}

// A unit of a row of type In: VE elements, widened to fp32 and rounded back once.
template <class In, bool VEC>
struct RowUnit;

template <class In>
struct RowUnit<In, true> {
  typedef u32x4 T;
  static constexpr int VE = In::VE;
  typedef typename std::conditional<In::ES == 2, OutBf16, OutF32>::type Out;
  __device__ static __forceinline__ T load(const T* p) { return ld16(p); }
  __device__ static __forceinline__ T load_kept(const T* p) { return *p; }  // read again soon: may stay in the caches
  __device__ static __forceinline__ void store(T* p, T v) { st16p<gci::kStoreDevNT>(p, v); }
  __device__ static __forceinline__ void widen(const T& v, float (&x)[VE]) { unpack<In>(v, x); }
  __device__ static __forceinline__ T narrow(const float (&x)[VE]) {
    const Words<Out, VE> r = pack<Out, VE>(x);
    return u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
  }
};

template <>
struct RowUnit<InBf16, false> {
  typedef uint16_t T;
  static constexpr int VE = 1;
  __device__ static __forceinline__ T load(const T* p) { return __builtin_nontemporal_load(p); }
  __device__ static __forceinline__ T load_kept(const T* p) { return *p; }
  __device__ static __forceinline__ void store(T* p, T v) { __builtin_nontemporal_store(v, p); }
  __device__ static __forceinline__ void widen(const T& v, float (&x)[1]) {
    x[0] = __uint_as_float(static_cast<uint32_t>(v) << 16);
  }
  __device__ static __forceinline__ T narrow(const float (&x)[1]) { return static_cast<T>(bf16_bits(x[0])); }
};

template <>
struct RowUnit<InF32, false> {
  typedef uint32_t T;
  static constexpr int VE = 1;
  __device__ static __forceinline__ T load(const T* p) { return __builtin_nontemporal_load(p); }
  __device__ static __forceinline__ T load_kept(const T* p) { return *p; }
  __device__ static __forceinline__ void store(T* p, T v) { __builtin_nontemporal_store(v, p); }
  __device__ static __forceinline__ void widen(const T& v, float (&x)[1]) { x[0] = __uint_as_float(v); }
  __device__ static __forceinline__ T narrow(const float (&x)[1]) { return __float_as_uint(x[0]); }
};

// Sum over a wavefront; every lane gets it.
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// Sum over LANES lanes (a wavefront or the workgroup), in an order fixed by the lanes.
// lds: one float per wavefront, free again when the call returns.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x, float* lds) {
  x = wave_sum(x);
  if constexpr (LANES > kWave) {
    const int w = threadIdx.x / kWave;
    if (threadIdx.x % kWave == 0) lds[w] = x;
    __syncthreads();
    float t = lds[0];
#pragma unroll
    for (int i = 1; i < LANES / kWave; ++i) t += lds[i];
    __syncthreads();
    x = t;
  }
  return x;
}

// ------------------------------------------------------------- 8-bit rows
//
// Block exponent e of the largest finite magnitude a (its fp32 bits): the
// smallest integer with a <= 448 * 2^e = 1.75 * 2^(e + 8), so e = E - 8 for
// a = 1.f * 2^E with 1.f <= 1.75, else E - 7: the carry out of the mantissa
// decides.  Clamped to [-117, 120]: below, every code times 2^e is still exact
// in bf16; 120 is what the largest finite a needs.
__device__ __forceinline__ int mx8_exponent(uint32_t abits) {
  const int e = static_cast<int>((abits + 0x1FFFFFu) >> 23) - 135;
  return min(max(e, -117), 120);
}

// Magnitude bits for the block maximum: infinities and NaN do not count.
__device__ __forceinline__ uint32_t mx8_magnitude(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// v * 2^-e, NaN for an infinity (e4m3 has none).  Exact: a product that
// leaves fp32's normal range is far below half of e4m3's smallest step.
__device__ __forceinline__ float mx8_scaled(float v, int e) {
  const float s = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  return (__float_as_uint(v) & 0x7FFFFFFFu) < 0x7F800000u ? v * s : __uint_as_float(0x7FC00000u);
}

// Four codes (nearest even; the hardware conversion, values within +-448) in one word.
__device__ __forceinline__ uint32_t mx8_codes(float a, float b, float c, float d) {
  int p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  p = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
  return static_cast<uint32_t>(p);
}

// Multiplier of a scale byte (0 stands for 0, 255 for infinity: the encoder writes neither).
__device__ __forceinline__ float mx8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

typedef float f32x2 __attribute__((ext_vector_type(2)));

// The values of four codes times the block's scale.
__device__ __forceinline__ void mx8_values(uint32_t codes, float scale, float (&v)[4]) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), true);
  v[0] = lo[0] * scale;
  v[1] = lo[1] * scale;
  v[2] = hi[0] * scale;
  v[3] = hi[1] * scale;
}

// Encodes one unit per lane of a row (unit u, VE values; 32 / VE consecutive
// lanes hold one block, so all of them call this together).  Lanes past the
// row's end pass ok = false.  row: the 8-bit row, n its values.
template <int VE>
__device__ __forceinline__ void mx8_encode(char* row, uint64_t n, uint64_t u, bool ok, const float (&v)[VE]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < VE; ++i) a = max(a, mx8_magnitude(v[i]));
  a = ok ? a : 0u;
#pragma unroll
  for (int o = 1; o < 32 / VE; o <<= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), o)));
  if (!ok) return;
  const int e = mx8_exponent(a);
  if constexpr (VE == 1) {
    row[u] = static_cast<char>(__builtin_amdgcn_cvt_pk_fp8_f32(mx8_scaled(v[0], e), 0.0f, 0, false));
  } else {
    uint32_t w[VE / 4];
#pragma unroll
    for (int i = 0; i < VE / 4; ++i)
      w[i] = mx8_codes(mx8_scaled(v[4 * i], e), mx8_scaled(v[4 * i + 1], e), mx8_scaled(v[4 * i + 2], e),
                       mx8_scaled(v[4 * i + 3], e));
    if constexpr (VE == 8) st8(row + 8 * u, u32x2{w[0], w[1]});
    else *reinterpret_cast<uint32_t*>(row + 4 * u) = w[0];
  }
  if (u % (32 / VE) == 0) row[n + u / (32 / VE)] = static_cast<char>(e + 127);
}

// Zero bytes behind the scales, up to the row's multiple of 16 (at most 15).
__device__ __forceinline__ void mx8_pad(char* row, uint64_t n, int lane) {
  const uint64_t used = n + (n + 31) / 32, end = (used + 15) / 16 * 16;
  if (used + lane < end) row[used + lane] = 0;
}

}  // namespace gcdev
