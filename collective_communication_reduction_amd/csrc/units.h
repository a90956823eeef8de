// Units of a row at any element alignment.  A unit is up to 16 bytes in one access,
// which the hardware takes at every address of the element's size, so one path
// serves every row length and offset.  The last unit of a row that is no multiple of
// it is moved inside the row and overlaps the one before: whole accesses only.
#pragma once

#include "rows.h"

namespace gcdev {

constexpr uint64_t kLine = 128;

template <class In, int N = In::VE>
struct AnyUnit {
  static constexpr int VE = N;
  static constexpr int NW = N * In::ES / 4;
  typedef uint32_t T __attribute__((ext_vector_type(NW)));
  typedef uint32_t TAny __attribute__((ext_vector_type(NW), aligned(2)));
  typedef typename std::conditional<In::ES == 2, OutBf16, OutF32>::type Out;
  typedef typename std::conditional<In::ES == 2, uint16_t, uint32_t>::type E;

  // First element of unit u in a row of n.  Rows shorter than a unit have one at 0.
  __device__ static __forceinline__ uint32_t start(uint32_t n, uint32_t u) { return gci::unit_start(n, VE, u); }
  // VE elements from s on, in a row of n; in a row shorter than that all of it, and `fill` (an element's bits) behind.
  // KEEP: read again soon, may stay in the caches.
  template <bool KEEP = false>
  __device__ static __forceinline__ T load(const char* row, uint32_t n, uint32_t s, uint32_t fill = 0) {
    const char* p = row + static_cast<uint64_t>(s) * In::ES;
    if (n < VE) return load_some(p, n, fill);
    if constexpr (KEEP) return *reinterpret_cast<const TAny*>(p);
    else return __builtin_nontemporal_load(reinterpret_cast<const TAny*>(p));
  }
  // The first k < VE elements at p.
  __device__ static __forceinline__ T load_some(const char* p, uint32_t k, uint32_t fill) {
    T v;
#pragma unroll
    for (int i = 0; i < NW; ++i) v[i] = In::ES == 2 ? fill << 16 | fill : fill;
    const E* e = reinterpret_cast<const E*>(p);
#pragma unroll
    for (uint32_t i = 0; i < VE - 1; ++i)
      if (i < k) {
        if constexpr (In::ES == 4) v[i] = e[i];
        else v[i / 2] = i % 2 ? (v[i / 2] & 0xFFFFu) | static_cast<uint32_t>(e[i]) << 16 : (v[i / 2] & 0xFFFF0000u) | e[i];
      }
    return v;
  }
  // VE elements from s on, or all of a shorter row.  through: to memory, past the L2; for rows that all start on a
  // line of memory (kLine).  Others share lines with their neighbours and are left to meet there.  Rows of 4092 fp32,
  // whole units but not lines, take less time so (lookup 619 us against 711, its gradient 1406 against 1668, 8 x 16384 rows).
  // Rows of whole lines take less through: the lookup of 8 x 16384 x 4096 bf16 from distinct rows 383 us against 410, its
  // gradient 584 against 650, dropout 501 against 520.  And a line that is written both ways takes a multiple (rows of
  // 4095 bf16: 0.8 TB/s where the units on a 16-byte boundary went through, 5.4 where none did).
  __device__ static __forceinline__ void store(char* row, uint32_t n, uint32_t s, T v, bool through) {
    char* p = row + static_cast<uint64_t>(s) * In::ES;
    if (n < VE) store_some(p, 0, n, v);
    else if (!through) *reinterpret_cast<TAny*>(p) = v;
    else if constexpr (NW == 4) st16p<gci::kStoreDevNT>(p, v);
    else __builtin_nontemporal_store(v, reinterpret_cast<T*>(p));
  }
  // Elements lo .. hi - 1 of a unit at p.
  __device__ static __forceinline__ void store_some(char* p, uint32_t lo, uint32_t hi, T v) {
    E* e = reinterpret_cast<E*>(p);
#pragma unroll
    for (uint32_t i = 0; i < VE; ++i)
      if (i >= lo && i < hi) e[i] = static_cast<E>(In::ES == 4 ? v[i] : v[i / 2] >> 16 * (i % 2));
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
