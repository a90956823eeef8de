// Root-mean-square norm of token rows with the residual's addition, and its
// backward pass, for gfx950.
//
//   forward   s = round(x + residual); rstd = (mean s^2 + eps)^(-1/2); y = s rstd w
//   backward  n = s rstd, d = dy w:  dx = rstd (d - n mean(d n)) + dsum,  dw = sum_t dy n
//
// Both read every input and write every output once: a row stays in registers
// between its sum and its outputs, so HBM bytes bound them.  Forward rows up to
// 64 x 2 units take one wavefront each (no barrier), longer ones a workgroup
// (4096 bf16, 512 units: 630 us with a workgroup's 2 units per lane, 641 with a
// wavefront's 8, for 8 x 16384 rows), and rows past a workgroup's registers are
// read a second time (from the caches, mostly).  Those 8 x 16384 rows: forward to
// 8-bit rows 623 us, 6.1 TB/s; backward 799 us, 5.4 TB/s (three streams read, one
// written), and 5 us for the weight gradient's partial sums.

#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace {

using namespace gcdev;

template <int P>
struct NormArgs {
  const char* x[P];
  const char* res[P];
  const char* w[P];
  char* sum[P];
  char* y[P];
  float* rstd[P];
  int64_t tok[P];
  int32_t tile0[P + 1];  // first workgroup of each rank
  uint32_t block0;       // first workgroup of this launch
  uint64_t H;            // elements per row
  uint64_t y_row;        // bytes per output row
  float eps;
  int32_t N;
  bool has_res, has_sum, has_rstd;
};

// s of one unit: x, or x + residual rounded to the row type.
template <class U>
__device__ __forceinline__ void residual_sum(const typename U::T& x, const typename U::T& r, bool has_res,
                                             float (&v)[U::VE], typename U::T& s) {
  U::widen(x, v);
  s = x;
  if (has_res) {
    float b[U::VE];
    U::widen(r, b);
#pragma unroll
    for (int e = 0; e < U::VE; ++e) v[e] += b[e];
    s = U::narrow(v);
    U::widen(s, v);
  }
}

// NV units per lane; a row's units lie LANES apart.
template <class In, bool VEC, bool MX, int NV, int LANES, int P>
__global__ void __launch_bounds__(kThreads) norm_kernel(const NormArgs<P> a) {
  typedef RowUnit<In, VEC> U;
  typedef typename U::T T;
  constexpr int VE = U::VE;
  __shared__ float lds[kThreads / kWave];
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int lane = threadIdx.x % LANES;
  const int64_t row = static_cast<int64_t>(block - a.tile0[rank]) * (kThreads / LANES) +
                      threadIdx.x / LANES;
  if (row >= a.tok[rank]) return;  // whole wavefronts (LANES == kThreads: never)
  const uint64_t units = a.H / VE;
  const T* x = reinterpret_cast<const T*>(a.x[rank]) + row * units;
  const T* r = reinterpret_cast<const T*>(a.res[rank]) + row * units;
  const T* w = reinterpret_cast<const T*>(a.w[rank]);
  T* sum = reinterpret_cast<T*>(a.sum[rank]) + row * units;
  T xv[NV], rv[NV], wv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint64_t u = min(static_cast<uint64_t>(lane + j * LANES), units - 1);  // clamped: no exec-masked load
    xv[j] = U::load(x + u);
    if (a.has_res) rv[j] = U::load(r + u);
    wv[j] = U::load_kept(w + u);
  }
  float v[NV][VE];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool ok = static_cast<uint64_t>(lane + j * LANES) < units;
    T s;
    residual_sum<U>(xv[j], rv[j], a.has_res, v[j], s);
    if (a.has_sum && ok) U::store(sum + lane + j * LANES, s);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float q = ok ? v[j][e] : 0.0f;  // both factors: 0 times an infinity in the row's last unit would be NaN
      ss = fmaf(q, q, ss);
    }
  }
  const float rs = 1.0f / sqrtf(lanes_sum<LANES>(ss, lds) / static_cast<float>(a.H) + a.eps);
  if (a.has_rstd && lane == 0) a.rstd[rank][row] = rs;
  char* yrow = a.y[rank] + row * a.y_row;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint64_t u = lane + j * LANES;
    const bool ok = u < units;
    float ww[VE];
    U::widen(wv[j], ww);
#pragma unroll
    for (int e = 0; e < VE; ++e) v[j][e] = v[j][e] * rs * ww[e];
    if constexpr (MX) mx8_encode<VE>(yrow, a.H, u, ok, v[j]);
    else if (ok) U::store(reinterpret_cast<T*>(yrow) + u, U::narrow(v[j]));
  }
  if constexpr (MX) mx8_pad(yrow, a.H, lane);
}

// Rows longer than a workgroup's registers: the sum's pass, then the output's.
// With sum_out the second pass reads what the first stored (the same lane).
template <class In, bool VEC, bool MX, int P>
__global__ void __launch_bounds__(kThreads) norm_long_kernel(const NormArgs<P> a) {
  typedef RowUnit<In, VEC> U;
  typedef typename U::T T;
  constexpr int VE = U::VE;
  __shared__ float lds[kThreads / kWave];
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int64_t row = block - a.tile0[rank];
  const uint64_t units = a.H / VE;
  const T* x = reinterpret_cast<const T*>(a.x[rank]) + row * units;
  const T* r = reinterpret_cast<const T*>(a.res[rank]) + row * units;
  const T* w = reinterpret_cast<const T*>(a.w[rank]);
  T* sum = reinterpret_cast<T*>(a.sum[rank]) + row * units;
  float ss = 0.0f;
  for (uint64_t u = threadIdx.x; u < units; u += kThreads) {
    T s, rr{};
    if (a.has_res) rr = U::load_kept(r + u);
    float v[VE];
    residual_sum<U>(U::load_kept(x + u), rr, a.has_res, v, s);
    if (a.has_sum) sum[u] = s;
#pragma unroll
    for (int e = 0; e < VE; ++e) ss = fmaf(v[e], v[e], ss);
  }
  const float rs = 1.0f / sqrtf(lanes_sum<kThreads>(ss, lds) / static_cast<float>(a.H) + a.eps);
  if (a.has_rstd && threadIdx.x == 0) a.rstd[rank][row] = rs;
  char* yrow = a.y[rank] + row * a.y_row;
  for (uint64_t u0 = 0; u0 < units; u0 += kThreads) {  // every lane, for the encoder
    const uint64_t u = u0 + threadIdx.x;
    const bool ok = u < units;
    const uint64_t c = ok ? u : units - 1;
    float v[VE], ww[VE];
    if (a.has_sum) {
      U::widen(sum[c], v);  // a clamped lane's value is not used
    } else {
      T s, rr{};
      if (a.has_res) rr = r[c];
      residual_sum<U>(x[c], rr, a.has_res, v, s);
    }
    U::widen(U::load_kept(w + c), ww);
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = v[e] * rs * ww[e];
    if constexpr (MX) mx8_encode<VE>(yrow, a.H, u, ok, v);
    else if (ok) U::store(reinterpret_cast<T*>(yrow) + u, U::narrow(v));
  }
  if constexpr (MX) mx8_pad(yrow, a.H, threadIdx.x);
}

// ------------------------------------------------------------- backward

template <int P>
struct NormBackwardArgs {
  const char* dy[P];
  const char* dsum[P];
  const char* sum[P];
  const char* w[P];
  const float* rstd[P];
  char* dx[P];
  float* dw[P];
  int64_t tok[P];
  int32_t tile0[P + 1];  // first block of each rank; block b leaves its partial in row b of `partial`
  uint32_t block0;       // first workgroup of this launch
  float* partial;
  uint64_t H;
  int64_t rows_per_block;
  int32_t N;
  bool has_dsum;
};

// One workgroup takes consecutive rows of one rank; each lane keeps the weight
// gradient of its own columns in registers over them and stores it once.
// Longer rows take more lanes rather than more units per lane: 20 units each
// left one wavefront per SIMD.
template <class In, bool VEC, int NV, int LANES, int P>
__global__ void __launch_bounds__(LANES) norm_backward_kernel(const NormBackwardArgs<P> a) {
  typedef RowUnit<In, VEC> U;
  typedef typename U::T T;
  constexpr int VE = U::VE;
  __shared__ float lds[LANES / kWave];
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int64_t first = static_cast<int64_t>(block - a.tile0[rank]) * a.rows_per_block;
  const int64_t last = min(first + a.rows_per_block, a.tok[rank]);
  const uint64_t units = a.H / VE;
  uint32_t c[NV];  // the lane's units; past the row's end its last unit again
  bool ok[NV];
  T wv[NV];
  float dw[NV][VE];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t u = threadIdx.x + j * LANES;
    ok[j] = u < units;
    c[j] = min(u, static_cast<uint32_t>(units - 1));
    wv[j] = U::load_kept(reinterpret_cast<const T*>(a.w[rank]) + c[j]);
#pragma unroll
    for (int e = 0; e < VE; ++e) dw[j][e] = 0.0f;
  }
  const T* const dy = reinterpret_cast<const T*>(a.dy[rank]);
  const T* const ds = reinterpret_cast<const T*>(a.dsum[rank]);
  const T* const sm = reinterpret_cast<const T*>(a.sum[rank]);
  // With few units per lane the next row's loads are in flight while this one's
  // sum goes round the workgroup (8 x 16384 x 4096 bf16: 25 us of 817 less).
  constexpr bool AHEAD = NV <= (LANES == 256 ? 2 : 1);  // else its registers would cost wavefronts
  T yn[NV], sn[NV], dn[NV];
  float rn = 0.0f;
  auto fetch = [&](int64_t row) {
    const T *const dy_row = dy + row * units, *const sm_row = sm + row * units, *const ds_row = ds + row * units;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      yn[j] = U::load(dy_row + c[j]);
      sn[j] = U::load(sm_row + c[j]);
      if (a.has_dsum) dn[j] = U::load(ds_row + c[j]);
    }
    rn = a.rstd[rank][row];
  };
  if (AHEAD && first < last) fetch(first);
  for (int64_t row = first; row < last; ++row) {
    T* dx = reinterpret_cast<T*>(a.dx[rank]) + row * units;
    if constexpr (!AHEAD) fetch(row);
    T yv[NV], sv[NV], dv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      yv[j] = yn[j];
      sv[j] = sn[j];
      dv[j] = dn[j];
    }
    const float rs = rn;
    if (AHEAD && row + 1 < last) fetch(row + 1);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float y[VE], n[VE], w[VE];
      U::widen(yv[j], y);
      U::widen(sv[j], n);
      U::widen(wv[j], w);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float g = y[e] * (n[e] * rs);
        dw[j][e] += g;
        dot = ok[j] ? fmaf(g, w[e], dot) : dot;  // not 0 * w: the clamped weight may be infinite
      }
    }
    const float mean = lanes_sum<LANES>(dot, lds) / static_cast<float>(a.H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float y[VE], n[VE], w[VE], d[VE];
      U::widen(yv[j], y);
      U::widen(sv[j], n);
      U::widen(wv[j], w);
      if (a.has_dsum) U::widen(dv[j], d);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float g = rs * (y[e] * w[e] - n[e] * rs * mean);
        d[e] = a.has_dsum ? g + d[e] : g;
      }
      if (ok[j]) U::store(dx + c[j], U::narrow(d));
    }
  }
  float* part = a.partial + static_cast<uint64_t>(block) * a.H;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (ok[j])
#pragma unroll
      for (int e = 0; e < VE; ++e) part[static_cast<uint64_t>(c[j]) * VE + e] = dw[j][e];
}

// Rows past a workgroup's registers: partial sums of the weight gradient live
// in the block's scratch row (each element read and written by one lane).
template <class In, bool VEC, int P>
__global__ void __launch_bounds__(kThreads) norm_backward_long_kernel(const NormBackwardArgs<P> a) {
  typedef RowUnit<In, VEC> U;
  typedef typename U::T T;
  constexpr int VE = U::VE;
  __shared__ float lds[kThreads / kWave];
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int64_t first = static_cast<int64_t>(block - a.tile0[rank]) * a.rows_per_block;
  const int64_t last = min(first + a.rows_per_block, a.tok[rank]);
  const uint64_t units = a.H / VE;
  const T* wt = reinterpret_cast<const T*>(a.w[rank]);
  float* part = a.partial + static_cast<uint64_t>(block) * a.H;
  for (int64_t row = first; row < last; ++row) {
    const T* dy = reinterpret_cast<const T*>(a.dy[rank]) + row * units;
    const T* ds = reinterpret_cast<const T*>(a.dsum[rank]) + row * units;
    const T* s = reinterpret_cast<const T*>(a.sum[rank]) + row * units;
    T* dx = reinterpret_cast<T*>(a.dx[rank]) + row * units;
    const float rs = a.rstd[rank][row];
    float dot = 0.0f;
    for (uint64_t u = threadIdx.x; u < units; u += kThreads) {
      float y[VE], n[VE], w[VE];
      U::widen(U::load_kept(dy + u), y);
      U::widen(U::load_kept(s + u), n);
      U::widen(U::load_kept(wt + u), w);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float g = y[e] * (n[e] * rs);
        part[u * VE + e] = row == first ? g : part[u * VE + e] + g;
        dot = fmaf(g, w[e], dot);
      }
    }
    const float mean = lanes_sum<kThreads>(dot, lds) / static_cast<float>(a.H);
    for (uint64_t u = threadIdx.x; u < units; u += kThreads) {
      float y[VE], n[VE], w[VE], d[VE];
      U::widen(dy[u], y);
      U::widen(s[u], n);
      U::widen(wt[u], w);
      if (a.has_dsum) U::widen(U::load(ds + u), d);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float g = rs * (y[e] * w[e] - n[e] * rs * mean);
        d[e] = a.has_dsum ? g + d[e] : g;
      }
      U::store(dx + u, U::narrow(d));
    }
  }
}

// dw of one rank: 64 columns per workgroup, each wavefront adds every fourth
// partial row of the rank's blocks, and the four sums are added in order.
template <int P>
__global__ void __launch_bounds__(kThreads) norm_weight_kernel(const NormBackwardArgs<P> a) {
  __shared__ float lds[kThreads / kWave][kWave];
  const int rank = blockIdx.y, w = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const uint64_t col = (static_cast<uint64_t>(a.block0) + blockIdx.x) * kWave + lane;
  constexpr int Q = kThreads / kWave;
  float acc = 0.0f;
  if (col < a.H) {
    const float* p = a.partial + col;
    int32_t b = a.tile0[rank] + w;
    const int32_t end = a.tile0[rank + 1];
    for (; b + 7 * Q < end; b += 8 * Q) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = p[static_cast<uint64_t>(b + i * Q) * a.H];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc += t[i];
    }
    for (; b < end; b += Q) acc += p[static_cast<uint64_t>(b) * a.H];
  }
  lds[w][lane] = acc;
  __syncthreads();
  if (w == 0 && col < a.H) a.dw[rank][col] = (lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane]);
}

// ------------------------------------------------------------- host side

// `blocks` workgroups in x, `ranks` in y.
template <class Kern, class A>
gc_status launch(Kern kernel, A& args, uint64_t blocks, hipStream_t stream, int threads = kThreads, int ranks = 1) {
  void* params[] = {&args};
  return gci::in_launches(blocks, threads, [&](uint32_t first, uint32_t n) {
    args.block0 = first;
    return gci::hip_status(hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(n, ranks), dim3(threads), params, 0, stream));
  });
}

uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

template <int P>
int32_t fill_tiles(int32_t (&tile0)[P + 1], int64_t (&tok)[P], const int64_t* tokens, int N, int64_t per) {
  int32_t run = 0;
  for (int s = 0; s < N; ++s) {
    tile0[s] = run;
    tok[s] = tokens[s];
    run += static_cast<int32_t>((tokens[s] + per - 1) / per);
  }
  for (int s = N; s <= P; ++s) tile0[s] = run;
  return run;
}

template <class In, bool VEC, bool MX, int P>
gc_status norm_impl(const gci::NormCall& c, NormArgs<P>& a) {
  const uint64_t units = c.hidden / RowUnit<In, VEC>::VE;
  const int64_t per = units <= 2 * kWave ? kThreads / kWave : 1;
  const int32_t g = fill_tiles<P>(a.tile0, a.tok, c.tokens, c.nranks, per);
  if (units <= 1 * kWave) return launch(norm_kernel<In, VEC, MX, 1, kWave, P>, a, g, c.stream);
  if (units <= 2 * kWave) return launch(norm_kernel<In, VEC, MX, 2, kWave, P>, a, g, c.stream);
  if (units <= 1 * kThreads) return launch(norm_kernel<In, VEC, MX, 1, kThreads, P>, a, g, c.stream);
  if (units <= 2 * kThreads) return launch(norm_kernel<In, VEC, MX, 2, kThreads, P>, a, g, c.stream);
  if (units <= 4 * kThreads) return launch(norm_kernel<In, VEC, MX, 4, kThreads, P>, a, g, c.stream);
  if (units <= 8 * kThreads) return launch(norm_kernel<In, VEC, MX, 8, kThreads, P>, a, g, c.stream);
  if constexpr (!VEC)
    if (units <= 32 * kThreads) return launch(norm_kernel<In, VEC, MX, 32, kThreads, P>, a, g, c.stream);
  return launch(norm_long_kernel<In, VEC, MX, P>, a, g, c.stream);
}

template <class In, int P>
gc_status norm_typed(const gci::NormCall& c) {
  NormArgs<P> a{};
  uint64_t m = c.hidden * In::ES;
  for (int s = 0; s < c.nranks; ++s) {
    a.x[s] = static_cast<const char*>(c.x[s]);
    a.w[s] = static_cast<const char*>(c.w[s]);
    a.y[s] = static_cast<char*>(c.y[s]);
    if (c.res) a.res[s] = static_cast<const char*>(c.res[s]);
    if (c.sum) a.sum[s] = static_cast<char*>(c.sum[s]);
    if (c.rstd) a.rstd[s] = c.rstd[s];
    if (c.tokens[s]) m |= addr(a.x[s]) | addr(a.res[s]) | addr(a.w[s]) | addr(a.sum[s]) | addr(a.y[s]);
  }
  a.H = c.hidden;
  a.y_row = c.y_t == GC_MX8 ? gci::mx8_row_bytes(c.hidden) : c.hidden * In::ES;
  a.eps = c.eps;
  a.N = c.nranks;
  a.has_res = c.res != nullptr;
  a.has_sum = c.sum != nullptr;
  a.has_rstd = c.rstd != nullptr;
  const bool vec = (m & 15) == 0, mx = c.y_t == GC_MX8;
  if (vec) return mx ? norm_impl<In, true, true, P>(c, a) : norm_impl<In, true, false, P>(c, a);
  return mx ? norm_impl<In, false, true, P>(c, a) : norm_impl<In, false, false, P>(c, a);
}

template <class In, bool VEC, int P>
gc_status norm_backward_impl(const gci::NormBackwardCall& c, NormBackwardArgs<P>& a) {
  const uint64_t units = c.hidden / RowUnit<In, VEC>::VE;
  const int32_t g = a.tile0[c.nranks];
  if (g) {
    gc_status st;
    if (units <= 256) st = launch(norm_backward_kernel<In, VEC, 1, 256, P>, a, g, c.stream, 256);
    else if (units <= 512) st = launch(norm_backward_kernel<In, VEC, 2, 256, P>, a, g, c.stream, 256);
    else if (units <= 1024) st = launch(norm_backward_kernel<In, VEC, 1, 1024, P>, a, g, c.stream, 1024);
    else if (units <= 2048) st = launch(norm_backward_kernel<In, VEC, 2, 1024, P>, a, g, c.stream, 1024);
    else if (!VEC && units <= 5 * 1024) st = launch(norm_backward_kernel<In, VEC, VEC ? 1 : 5, 1024, P>, a, g, c.stream, 1024);
    else st = launch(norm_backward_long_kernel<In, VEC, P>, a, g, c.stream);
    if (st != GC_OK) return st;
  }
  return launch(norm_weight_kernel<P>, a, (c.hidden + kWave - 1) / kWave, c.stream, kThreads, c.nranks);
}

template <class In, int P>
gc_status norm_backward_typed(const gci::NormBackwardCall& c) {
  NormBackwardArgs<P> a{};
  uint64_t m = c.hidden * In::ES;
  for (int s = 0; s < c.nranks; ++s) {
    a.dy[s] = static_cast<const char*>(c.dy[s]);
    a.sum[s] = static_cast<const char*>(c.sum[s]);
    a.w[s] = static_cast<const char*>(c.w[s]);
    a.rstd[s] = c.rstd[s];
    a.dx[s] = static_cast<char*>(c.dx[s]);
    a.dw[s] = c.dw[s];
    if (c.dsum) a.dsum[s] = static_cast<const char*>(c.dsum[s]);
    if (c.tokens[s]) m |= addr(a.dy[s]) | addr(a.dsum[s]) | addr(a.sum[s]) | addr(a.w[s]) | addr(a.dx[s]);
  }
  fill_tiles<P>(a.tile0, a.tok, c.tokens, c.nranks, c.rows_per_block);
  a.partial = c.partial;
  a.H = c.hidden;
  a.rows_per_block = c.rows_per_block;
  a.N = c.nranks;
  a.has_dsum = c.dsum != nullptr;
  return (m & 15) == 0 ? norm_backward_impl<In, true, P>(c, a) : norm_backward_impl<In, false, P>(c, a);
}

}  // namespace

namespace gci {

gc_status launch_rms_norm(const NormCall& c) {
  if (c.t == GC_BF16) return c.nranks <= 8 ? norm_typed<InBf16, 8>(c) : norm_typed<InBf16, 64>(c);
  return c.nranks <= 8 ? norm_typed<InF32, 8>(c) : norm_typed<InF32, 64>(c);
}

gc_status launch_rms_norm_backward(const NormBackwardCall& c) {
  if (c.t == GC_BF16) return c.nranks <= 8 ? norm_backward_typed<InBf16, 8>(c) : norm_backward_typed<InBf16, 64>(c);
  return c.nranks <= 8 ? norm_backward_typed<InF32, 8>(c) : norm_backward_typed<InF32, 64>(c);
}

}  // namespace gci
