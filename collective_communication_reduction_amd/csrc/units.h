// Units of a row at any element alignment: 16 bytes in one access (the hardware
// takes them at every address of the element's size; an odd start costs a 17th
// of the lines more), and the row's last unit element by element where it is
// short.  One path therefore serves every row length and offset.
#pragma once

#include "rows.h"

namespace gcdev {

typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <class In>
struct AnyUnit {
  static constexpr int VE = In::VE;
  typedef typename std::conditional<In::ES == 2, OutBf16, OutF32>::type Out;
  typedef typename std::conditional<In::ES == 2, uint16_t, uint32_t>::type E;

  // Elements 8 u (4 u) and on of a row of n, `fill` past its end.  row + n is never passed.
  // KEEP: read again soon, may stay in the caches.
  template <bool KEEP = false>
  __device__ static __forceinline__ u32x4 load(const char* row, uint64_t n, uint64_t u, uint32_t fill) {
    const char* p = row + u * 16;
    if ((u + 1) * VE <= n) {
      const u32x4_any* q = reinterpret_cast<const u32x4_any*>(p);
      if constexpr (KEEP) return *q;
      else return __builtin_nontemporal_load(q);
    }
    return load_tail(p, u * VE < n ? static_cast<int>(n - u * VE) : 0, fill);
  }
  // A whole unit.
  __device__ static __forceinline__ u32x4 load_whole(const char* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
  }
  // The first k < VE elements at p; fill: one element's bits, on both halves of a word for 2-byte elements.
  __device__ static __forceinline__ u32x4 load_tail(const char* p, int k, uint32_t fill) {
    u32x4 v = {fill, fill, fill, fill};
    const E* e = reinterpret_cast<const E*>(p);
#pragma unroll
    for (int i = 0; i < VE - 1; ++i)
      if (i < k) {
        if constexpr (In::ES == 4) v[i] = e[i];
        else v[i / 2] = i % 2 ? (v[i / 2] & 0xFFFFu) | static_cast<uint32_t>(e[i]) << 16 : (v[i / 2] & 0xFFFF0000u) | e[i];
      }
    return v;
  }
  // The first min(VE, n - VE u) of the unit's elements; nothing past the row's end.
  __device__ static __forceinline__ void store(char* row, uint64_t n, uint64_t u, u32x4 v) {
    char* p = row + u * 16;
    if ((u + 1) * VE <= n) {
      st16p<gci::kStoreDevNT>(p, v);
      return;
    }
    E* e = reinterpret_cast<E*>(p);
#pragma unroll
    for (int i = 0; i < VE - 1; ++i)
      if (u * VE + i < n) e[i] = static_cast<E>(In::ES == 4 ? v[i] : v[i / 2] >> 16 * (i % 2));
  }
  __device__ static __forceinline__ void widen(const u32x4& v, float (&x)[VE]) { unpack<In>(v, x); }
  __device__ static __forceinline__ u32x4 narrow(const float (&x)[VE]) {
    const Words<Out, VE> r = pack<Out, VE>(x);
    return u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
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
