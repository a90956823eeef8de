// Units of a row at any element alignment: up to 16 bytes in one access, which the
// hardware takes at every address of the element's size, and the row's last unit
// element by element where it is short.  One path therefore serves every row
// length and offset (rows of 31999 bf16 logits read at 94 % of 32000's rate).
#pragma once

#include "rows.h"

namespace gcdev {

template <class In, int N = In::VE>
struct AnyUnit {
  static constexpr int VE = N;
  static constexpr int NW = N * In::ES / 4;
  typedef uint32_t T __attribute__((ext_vector_type(NW)));
  typedef uint32_t TAny __attribute__((ext_vector_type(NW), aligned(2)));
  typedef typename std::conditional<In::ES == 2, OutBf16, OutF32>::type Out;
  typedef typename std::conditional<In::ES == 2, uint16_t, uint32_t>::type E;

  // Elements VE u and on of a row of n; `fill` (an element's bits) past its end, where nothing is read.
  // KEEP: read again soon, may stay in the caches.
  template <bool KEEP = false>
  __device__ static __forceinline__ T load(const char* row, uint64_t n, uint64_t u, uint32_t fill = 0) {
    const char* p = row + u * (VE * In::ES);
    if ((u + 1) * VE <= n) {
      if constexpr (KEEP) return *reinterpret_cast<const TAny*>(p);
      else return __builtin_nontemporal_load(reinterpret_cast<const TAny*>(p));
    }
    const int k = u * VE < n ? static_cast<int>(n - u * VE) : 0;
    const E* e = reinterpret_cast<const E*>(p);
    T v;
#pragma unroll
    for (int i = 0; i < NW; ++i) v[i] = In::ES == 2 ? fill << 16 | fill : fill;
#pragma unroll
    for (int i = 0; i < VE - 1; ++i)
      if (i < k) {
        if constexpr (In::ES == 4) v[i] = e[i];
        else v[i / 2] = i % 2 ? (v[i / 2] & 0xFFFFu) | static_cast<uint32_t>(e[i]) << 16 : (v[i / 2] & 0xFFFF0000u) | e[i];
      }
    return v;
  }
  // Stores what the row holds of the unit.  On a boundary of its size a unit goes through to memory; elsewhere
  // neighbouring units share lines, and those are left to meet in the L2.
  __device__ static __forceinline__ void store(char* row, uint64_t n, uint64_t u, T v) {
    char* p = row + u * (VE * In::ES);
    if ((u + 1) * VE <= n) {
      if (reinterpret_cast<uintptr_t>(p) % sizeof(T)) *reinterpret_cast<TAny*>(p) = v;
      else if constexpr (NW == 4) st16p<gci::kStoreDevNT>(p, v);
      else __builtin_nontemporal_store(v, reinterpret_cast<T*>(p));
      return;
    }
    E* e = reinterpret_cast<E*>(p);
#pragma unroll
    for (int i = 0; i < VE - 1; ++i)
      if (u * VE + i < n) e[i] = static_cast<E>(In::ES == 4 ? v[i] : v[i / 2] >> 16 * (i % 2));
  }
  __device__ static __forceinline__ void widen(const T& v, float (&x)[VE]) {
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      if constexpr (In::ES == 4) x[i] = __uint_as_float(v[i]);
      else x[i] = __uint_as_float(i % 2 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
    }
  }
  __device__ static __forceinline__ T narrow(const float (&x)[VE]) {
    const Words<Out, VE> r = pack<Out, VE>(x);
    T v;
#pragma unroll
    for (int i = 0; i < NW; ++i) v[i] = r.w[i];
    return v;
  }
};

// Workgroups of each rank in one index space: first[r] the first of rank r, `per` rows each.
template <int P>
bool fill_blocks(int32_t (&first)[P + 1], const int64_t* rows, int N, uint64_t per, uint64_t slices = 1) {
  uint64_t run = 0;
  for (int s = 0; s < N; ++s) {
    first[s] = static_cast<int32_t>(run);
    run += (static_cast<uint64_t>(rows[s]) * slices + per - 1) / per;
    if (run >= (uint64_t(1) << 31)) return false;
  }
  for (int s = N; s <= P; ++s) first[s] = static_cast<int32_t>(run);
  return true;
}

// `blocks` workgroups of one kernel; args.block0 numbers the launch's first.
template <class Kern, class A>
gc_status launch_blocks(Kern kernel, A& args, uint64_t blocks, int threads, hipStream_t stream) {
  void* params[] = {&args};
  return gci::in_launches(blocks, threads, [&](uint32_t first, uint32_t n) {
    args.block0 = first;
    return gci::hip_status(hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(n), dim3(threads), params, 0, stream));
  });
}

}  // namespace gcdev
