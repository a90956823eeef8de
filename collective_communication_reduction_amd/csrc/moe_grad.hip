// Gradient of the MoE combine for gfx950: out[t] = sum_k w_k y[dest_k] gives
// dy[dest_k] = w_k dout[t] and dw_k = <dout[t], y[dest_k]>.  Each token's dout
// row is read once and serves its K routes; every expert row is read and
// written once.  HBM bytes bound it: (1 + 2K) rows per token.  A wavefront (or
// fewer lanes, for short rows) takes one token; the dots stay in registers over
// the row and are summed across the lanes once.  8 x 16384 tokens of 4096 bf16,
// top-2: 956 us, 5.6 TB/s, its expert rows scattered over 64 blocks.

#include <type_traits>

#include "rows.h"

namespace {

using namespace gcdev;

constexpr int kGradU = 8;      // units per lane per step: a 4096-wide bf16 row at once (5 % less than with 4, 8 x 16384 tokens)
constexpr int kMaxTopk = 8;

template <int P>
struct CombineBackwardArgs {
  const char* dout[P];
  const char* y[P];
  char* dy[P];
  const int2* dest[P];
  const float* w[P];
  float* dw[P];
  int64_t rows[P];
  int64_t tok[P];
  int32_t tile0[P + 1];  // first workgroup of each rank
  uint32_t block0;       // first workgroup of this launch
  uint64_t R;            // units per row
  int32_t N, K, lanes_log2;
};

template <class In, bool VEC, int KT, int P>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const CombineBackwardArgs<P> a) {
  typedef RowUnit<In, VEC> U;
  typedef typename U::T T;
  constexpr int VE = U::VE;
  constexpr int KM = KT > 0 ? KT : kMaxTopk;
  const int K = KT > 0 ? KT : a.K;
  const int S = 1 << a.lanes_log2;
  const int lane = threadIdx.x & (S - 1);
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int64_t t = static_cast<int64_t>(block - a.tile0[rank]) * (kThreads >> a.lanes_log2) +
                    (threadIdx.x >> a.lanes_log2);
  const bool live = t < a.tok[rank];
  const int64_t tc = live ? t : a.tok[rank] - 1;  // the last token again: reads stay inside, nothing is written
  const T* dout = reinterpret_cast<const T*>(a.dout[rank]) + static_cast<uint64_t>(tc) * a.R;
  const T* y[KM];
  T* dy[KM];
  float w[KM], dot[KM];
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    dot[k] = 0.0f;
    y[k] = nullptr;
    dy[k] = nullptr;
    w[k] = 0.0f;
    if (k < K) {
      const int2 p = a.dest[rank][tc * K + k];
      const bool in = p.x >= 0 && p.x < a.N;
      const int q = in ? p.x : 0;
      if (in && p.y >= 0 && p.y < a.rows[q]) {
        y[k] = reinterpret_cast<const T*>(a.y[q]) + static_cast<uint64_t>(p.y) * a.R;
        dy[k] = reinterpret_cast<T*>(a.dy[q]) + static_cast<uint64_t>(p.y) * a.R;
      }
      w[k] = a.w[rank][tc * K + k];
    }
  }
  for (uint64_t c = lane; c < a.R; c += static_cast<uint64_t>(kGradU) * S) {
    T g[kGradU];
#pragma unroll
    for (int j = 0; j < kGradU; ++j) {
      const uint64_t cj = c + static_cast<uint64_t>(j) * S;
      g[j] = U::load(dout + (cj < a.R ? cj : c));
    }
    T v[KT > 0 ? KT : 1][kGradU];
    if constexpr (KT > 0) {
#pragma unroll
      for (int k = 0; k < KT; ++k)
        if (y[k]) {
#pragma unroll
          for (int j = 0; j < kGradU; ++j) {
            const uint64_t cj = c + static_cast<uint64_t>(j) * S;
            v[k][j] = U::load(y[k] + (cj < a.R ? cj : c));
          }
        }
    }
#pragma unroll
    for (int k = 0; k < KM; ++k) {
      if (!y[k]) continue;
      if constexpr (KT == 0) {
#pragma unroll
        for (int j = 0; j < kGradU; ++j) {
          const uint64_t cj = c + static_cast<uint64_t>(j) * S;
          v[0][j] = U::load(y[k] + (cj < a.R ? cj : c));
        }
      }
#pragma unroll
      for (int j = 0; j < kGradU; ++j) {
        const uint64_t cj = c + static_cast<uint64_t>(j) * S;
        if (cj >= a.R) continue;
        float x[VE], z[VE], o[VE];
        U::widen(g[j], x);
        U::widen(v[KT > 0 ? k : 0][j], z);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          dot[k] = fmaf(x[e], z[e], dot[k]);
          o[e] = w[k] * x[e];
        }
        if (live) U::store(dy[k] + cj, U::narrow(o));
      }
    }
  }
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    if (k >= K) break;
    float d = dot[k];
    for (int o = S >> 1; o > 0; o >>= 1) d += __shfl_xor(d, o);
    if (lane == 0 && live) a.dw[rank][t * K + k] = d;
  }
}

template <class In, bool VEC, int P>
gc_status combine_backward_impl(const gci::MoeCombineBackwardCall& c, CombineBackwardArgs<P>& a) {
  a.R = c.hidden / RowUnit<In, VEC>::VE;
  a.lanes_log2 = 0;
  while (a.lanes_log2 < 6 && (uint64_t(1) << a.lanes_log2) * kGradU < a.R) ++a.lanes_log2;
  const int64_t per = kThreads >> a.lanes_log2;
  int32_t run = 0;
  for (int s = 0; s < c.nranks; ++s) {
    a.tile0[s] = run;
    run += static_cast<int32_t>((c.tokens[s] + per - 1) / per);
  }
  for (int s = c.nranks; s <= P; ++s) a.tile0[s] = run;
  void* params[] = {&a};
  const void* k = c.topk == 1   ? reinterpret_cast<const void*>(combine_backward_kernel<In, VEC, 1, P>)
                  : c.topk == 2 ? reinterpret_cast<const void*>(combine_backward_kernel<In, VEC, 2, P>)
                                : reinterpret_cast<const void*>(combine_backward_kernel<In, VEC, 0, P>);
  return gci::in_launches(run, kThreads, [&](uint32_t first, uint32_t blocks) {
    a.block0 = first;
    return gci::hip_status(hipLaunchKernel(k, dim3(blocks), dim3(kThreads), params, 0, c.stream));
  });
}

template <class In, int P>
gc_status combine_backward_typed(const gci::MoeCombineBackwardCall& c) {
  CombineBackwardArgs<P> a{};
  uint64_t m = c.hidden * In::ES;
  for (int s = 0; s < c.nranks; ++s) {
    a.dout[s] = static_cast<const char*>(c.dout[s]);
    a.y[s] = static_cast<const char*>(c.y[s]);
    a.dy[s] = static_cast<char*>(c.dy[s]);
    a.dest[s] = reinterpret_cast<const int2*>(c.dest[s]);
    a.w[s] = c.weights[s];
    a.dw[s] = c.dweights[s];
    a.rows[s] = c.y_rows[s];
    a.tok[s] = c.tokens[s];
    if (c.tokens[s]) m |= reinterpret_cast<uint64_t>(a.dout[s]);
    if (c.y_rows[s]) m |= reinterpret_cast<uint64_t>(a.y[s]) | reinterpret_cast<uint64_t>(a.dy[s]);
  }
  a.N = c.nranks;
  a.K = c.topk;
  return (m & 15) == 0 ? combine_backward_impl<In, true, P>(c, a) : combine_backward_impl<In, false, P>(c, a);
}

}  // namespace

namespace gci {

gc_status launch_moe_combine_backward(const MoeCombineBackwardCall& c) {
  if (c.t == GC_BF16)
    return c.nranks <= 8 ? combine_backward_typed<InBf16, 8>(c) : combine_backward_typed<InBf16, 64>(c);
  return c.nranks <= 8 ? combine_backward_typed<InF32, 8>(c) : combine_backward_typed<InF32, 64>(c);
}

}  // namespace gci
