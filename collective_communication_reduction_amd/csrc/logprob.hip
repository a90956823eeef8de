// Log probabilities of given tokens, the entropy of their distribution, its most
// likely tokens, and the gradient of the logits, for gfx950.
//
//   z = scale * x,  m = max x,  d = scale * (x - m),  S = sum e^d,  U = sum d e^d
//   lse = scale * m + log S,  log p = d - log S,  entropy = log S - U / S
//   dx = scale * (dlogprob * ([target] - p) - dentropy * p * (log p + entropy))
//
// One pass over a row keeps the running maximum m and rescales S and U when it
// grows; sums are fp32.

#include <type_traits>

#include "units.h"

namespace {

using namespace gcdev;

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kFarBelow = -1e30f;   // in place of -inf where it meets a factor of 0

template <int P>
struct LogprobArgs {
  const char* logits[P];
  const int32_t* targets[P];
  float* logprob[P];
  float* entropy[P];
  float* lse[P];
  int32_t* top_ids[P];
  float* top_logprob[P];
  const float* dlogprob[P];
  const float* dentropy[P];
  char* dlogits[P];
  int32_t tile0[P + 1];
  uint32_t block0;
  int32_t N;
  int32_t top;
  float scale;
  uint64_t V;
  uint64_t stride;
};

// Natural exponential; below e^-87 it flushes to 0.
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2E); }

// Unit u of a row of n logits, -inf past its end.
template <class In>
__device__ __forceinline__ u32x4 load_own(const char* row, uint64_t n, uint64_t u) {
  typedef AnyUnit<In> U;
  const uint32_t left = static_cast<uint32_t>(min<uint64_t>(U::VE, n > u * U::VE ? n - u * U::VE : 0));
  return U::load(row + u * 16, left, 0, In::ES == 2 ? 0xFF80u : 0xFF800000u);
}
template <class In>
__device__ __forceinline__ void store_own(char* row, uint64_t n, uint64_t u, u32x4 v) {
  typedef AnyUnit<In> U;
  U::store(row + u * 16, static_cast<uint32_t>(min<uint64_t>(U::VE, n - u * U::VE)), 0, v, n * In::ES % kLine == 0);
}

// Sums of a set of logits relative to its maximum.
struct Stat {
  float m, s, u;
};

// c.s and c.u of values at maximum c.m, taken to a maximum of m.
__device__ __forceinline__ void raise(Stat& c, float m, float scale) {
  const float d = c.m == m ? 0.0f : fmaxf(scale * (c.m - m), kFarBelow);
  const float f = exp_of(d);
  c.u = f * fmaf(c.s, d, c.u);
  c.s *= f;
  c.m = m;
}

__device__ __forceinline__ Stat join(Stat a, Stat b, float scale) {
  const float m = fmaxf(a.m, b.m);
  raise(a, m, scale);
  raise(b, m, scale);
  return Stat{m, a.s + b.s, a.u + b.u};
}

template <int VE>
__device__ __forceinline__ void add(Stat& c, const float (&x)[VE], float scale) {
  float m = c.m;
#pragma unroll
  for (int e = 0; e < VE; ++e) m = fmaxf(m, x[e]);
  if (m > c.m) raise(c, m, scale);
  const float base = m == kNegInf ? 0.0f : m;
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const float d = scale * (x[e] - base), p = exp_of(d);
    c.s += p;
    c.u = fmaf(p, fmaxf(d, kFarBelow), c.u);
  }
}

// The workgroup's Stat; every lane gets it.
__device__ __forceinline__ Stat block_stat(Stat c, float scale, Stat* lds) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1)
    c = join(c, Stat{__shfl_xor(c.m, o), __shfl_xor(c.s, o), __shfl_xor(c.u, o)}, scale);
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = c;
  __syncthreads();
  c = lds[0];
  for (int w = 1; w < kThreads / kWave; ++w) c = join(c, lds[w], scale);
  __syncthreads();
  return c;
}

// Order of the alternatives: by value, then the lowest token first; 0 is below every value.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t id) {
  const uint32_t b = __float_as_uint(x + 0.0f);   // -0 counts as 0
  const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
  return x != x ? 0 : static_cast<uint64_t>(k) << 32 | (0xFFFFFFFFu - id);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int o) {
  const uint32_t lo = __shfl_xor(static_cast<uint32_t>(x), o), hi = __shfl_xor(static_cast<uint32_t>(x >> 32), o);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

__device__ __forceinline__ uint64_t block_max(uint64_t x, uint64_t* lds) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) {
    const uint64_t y = shfl_xor64(x, o);
    x = x > y ? x : y;
  }
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = x;
  __syncthreads();
  x = lds[0];
  for (int w = 1; w < kThreads / kWave; ++w) x = x > lds[w] ? x : lds[w];
  __syncthreads();
  return x;
}

// What the gradient of one row needs.
struct RowGrad {
  float m, log_s, inv_s, entropy, dlp, dent, scale;
  int32_t target;
  bool empty;
};

// log p of one logit and its gradient.
template <bool ENT>
__device__ __forceinline__ float grad_of(const RowGrad& g, float d, bool target) {
  const float p = exp_of(d) * g.inv_s;
  float v = g.dlp * ((target ? 1.0f : 0.0f) - p);
  if constexpr (ENT) v -= g.dent * (p * (fmaxf(d - g.log_s, kFarBelow) + g.entropy));
  return g.empty ? 0.0f : v * g.scale;
}

template <class In, bool ENT>
__device__ __forceinline__ void put_grads(const RowGrad& g, const char* row, char* out, uint64_t V, uint64_t stride) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE;
  const uint64_t units = (stride + VE - 1) / VE;
  for (uint64_t u = threadIdx.x; u < units; u += kThreads) {
    float x[VE];
    U::widen(load_own<In>(row, V, u), x);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const uint64_t i = u * VE + e;
      x[e] = i < V ? grad_of<ENT>(g, g.scale * (x[e] - g.m), static_cast<int64_t>(i) == g.target) : 0.0f;
    }
    store_own<In>(out, stride, u, U::narrow(x));
  }
}

template <class In, int P>
__global__ void __launch_bounds__(kThreads) logprob_kernel(const LogprobArgs<P> a) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE;
  __shared__ Stat stats[kThreads / kWave];
  __shared__ uint64_t best[kThreads / kWave];
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int64_t r = block - a.tile0[rank];
  const char* row = a.logits[rank] + static_cast<uint64_t>(r) * a.stride * In::ES;
  const uint64_t units = (a.V + VE - 1) / VE;
  Stat c{kNegInf, 0.0f, 0.0f};
  for (uint64_t u = threadIdx.x; u < units; u += kThreads) {
    float x[VE];
    U::widen(load_own<In>(row, a.V, u), x);
    add<VE>(c, x, a.scale);
  }
  c = block_stat(c, a.scale, stats);
  const bool empty = c.s == 0.0f;
  const float log_s = empty ? 0.0f : logf(c.s);
  const float m = empty ? 0.0f : c.m;
  const float entropy = empty ? 0.0f : log_s - c.u / c.s;
  int32_t target = a.targets[rank] ? a.targets[rank][r] : -1;
  if (static_cast<uint32_t>(target) >= a.V) target = -1;
  if (threadIdx.x == 0) {
    if (a.lse[rank]) a.lse[rank][r] = empty ? kNegInf : a.scale * m + log_s;
    if (a.entropy[rank]) a.entropy[rank][r] = entropy;
    if (a.logprob[rank])
      a.logprob[rank][r] = target < 0 ? 0.0f : empty ? kNegInf : a.scale * (In::one(row, target) - m) - log_s;
  }
  uint64_t prev = ~uint64_t(0);
  for (int k = 0; k < a.top; ++k) {
    uint64_t b = 0;
    for (uint64_t u = threadIdx.x; u < units; u += kThreads) {
      float x[VE];
      U::widen(load_own<In>(row, a.V, u), x);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const uint64_t i = u * VE + e, key = i < a.V ? order_key(x[e], static_cast<uint32_t>(i)) : 0;
        if (key < prev && key > b) b = key;
      }
    }
    prev = block_max(b, best);
    if (threadIdx.x == 0) {
      const int64_t at = r * a.top + k;
      const int32_t id = prev ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(prev)) : -1;
      a.top_ids[rank][at] = id;
      a.top_logprob[rank][at] = id < 0 || empty ? (c.s != c.s ? c.s : kNegInf) : a.scale * (In::one(row, id) - m) - log_s;
    }
  }
  if (!a.dlogits[rank]) return;
  __syncthreads();   // dlogits may be logits: single values of the row were read above
  const RowGrad g{m, log_s, 1.0f / c.s, entropy, target < 0 ? 0.0f : a.dlogprob[rank][r],
                  a.dentropy[rank] ? a.dentropy[rank][r] : 0.0f, a.scale, target, empty};
  char* out = a.dlogits[rank] + static_cast<uint64_t>(r) * a.stride * In::ES;
  if (a.dentropy[rank]) put_grads<In, true>(g, row, out, a.V, a.stride);
  else put_grads<In, false>(g, row, out, a.V, a.stride);
}

// The gradient from the saved lse and entropy: p = e^(z - lse).
template <class In, bool ENT, int P>
__global__ void __launch_bounds__(kThreads) logprob_backward_kernel(const LogprobArgs<P> a) {
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int64_t r = block - a.tile0[rank];
  const float lse = a.lse[rank][r];
  int32_t target = a.targets[rank][r];
  if (static_cast<uint32_t>(target) >= a.V) target = -1;
  const RowGrad g{0.0f, 0.0f, 1.0f, ENT ? a.entropy[rank][r] : 0.0f, target < 0 ? 0.0f : a.dlogprob[rank][r],
            ENT ? a.dentropy[rank][r] : 0.0f, a.scale, target, lse == kNegInf};
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE;
  const uint64_t off = static_cast<uint64_t>(r) * a.stride * In::ES;
  const char* row = a.logits[rank] + off;
  char* out = a.dlogits[rank] + off;
  const uint64_t units = (a.stride + VE - 1) / VE;
  for (uint64_t u = threadIdx.x; u < units; u += kThreads) {
    float x[VE];
    U::widen(load_own<In>(row, a.V, u), x);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const uint64_t i = u * VE + e;
      x[e] = i < a.V ? grad_of<ENT>(g, fmaf(a.scale, x[e], -lse), static_cast<int64_t>(i) == target) : 0.0f;
    }
    store_own<In>(out, a.stride, u, U::narrow(x));
  }
}

template <class In, int P>
gc_status logprob_typed(const gci::LogprobCall& c, bool backward) {
  LogprobArgs<P> a{};
  for (int s = 0; s < c.nranks; ++s) {
    a.logits[s] = static_cast<const char*>(c.logits[s]);
    if (c.targets) a.targets[s] = c.targets[s];
    if (c.logprob) a.logprob[s] = c.logprob[s];
    if (c.entropy) a.entropy[s] = c.entropy[s];
    if (c.lse) a.lse[s] = c.lse[s];
    if (c.top) a.top_ids[s] = c.top_ids[s];
    if (c.top) a.top_logprob[s] = c.top_logprob[s];
    if (c.dlogprob) a.dlogprob[s] = c.dlogprob[s];
    if (c.dentropy) a.dentropy[s] = c.dentropy[s];
    if (c.dlogits) a.dlogits[s] = static_cast<char*>(c.dlogits[s]);
  }
  fill_blocks<P>(a.tile0, c.tokens, c.nranks, 1);
  a.N = c.nranks;
  a.top = c.top;
  a.scale = c.scale;
  a.V = c.vocab;
  a.stride = c.stride;
  const int32_t g = a.tile0[c.nranks];
  if (!backward) return launch_blocks(logprob_kernel<In, P>, a, g, kThreads, c.stream);
  return c.dentropy ? launch_blocks(logprob_backward_kernel<In, true, P>, a, g, kThreads, c.stream)
                    : launch_blocks(logprob_backward_kernel<In, false, P>, a, g, kThreads, c.stream);
}

gc_status logprob_any(const gci::LogprobCall& c, bool backward) {
  if (c.t == GC_BF16) return c.nranks <= 8 ? logprob_typed<InBf16, 8>(c, backward) : logprob_typed<InBf16, 64>(c, backward);
  return c.nranks <= 8 ? logprob_typed<InF32, 8>(c, backward) : logprob_typed<InF32, 64>(c, backward);
}

}  // namespace

namespace gci {

gc_status launch_token_logprob(const LogprobCall& c) { return logprob_any(c, false); }
gc_status launch_token_logprob_backward(const LogprobCall& c) { return logprob_any(c, true); }

}  // namespace gci
