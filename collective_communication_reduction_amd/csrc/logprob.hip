// Log probabilities of given tokens, the entropy of their distribution, its most
// likely tokens, and the gradient of the logits, for gfx950.
//
//   t = x scale log2(e) - r,  S = sum 2^t,  U = sum t 2^t      (r: the largest x times scale log2(e), rounded)
//   lse = ln2 (r + log2 S),  log p = ln2 (t - log2 S),  entropy = ln2 (log2 S - U / S)
//   dx = scale (dlogprob ([target] - p) - dentropy p (log p + entropy))
//
// One pass: a group of lanes (a wavefront or a workgroup) holds a row in registers,
// each lane takes its own values' maximum and sums relative to it, and the lanes'
// sums are joined at the end.  Longer rows go through the registers in tiles, and
// only their gradient reads them again.  HBM bytes bound it, with about ten vector
// operations a value, four of them the exponential's quarter rate, close behind:
// 8 x 4096 rows of 32000 bf16 take 316 us for the sums (6.6 TB/s), 729 with the
// gradient (5.8 TB/s, read and written); 4 x 2048 rows with five alternatives 108
// (4.9 TB/s); the gradient from a saved lse of 2 x 1024 x 131072 178 (6.0 TB/s).
// All times here are of calls queued one after the other on one card (short ones
// replayed from a graph); others differ by up to 5 %, and kernels that a profiler
// runs one at a time take up to a quarter longer.

#include <type_traits>

#include "units.h"

namespace {

using namespace gcdev;

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_huge_valf();
constexpr float kFarBelow = -1e30f;   // in place of -inf where it meets a factor of 0
constexpr float kNoneBelow = -256.0f; // from here on 2^t and e^t are 0
constexpr float kLargeFactor = 0x1p100f;
constexpr float kLargest = 0x1p14f;   // of r: its rounding moves t by 2^-11 at most, p by less than half of bf16's rounding

constexpr int kMostParts = gci::kLogprobParts;

enum Mode { kStats, kTop, kGrad };    // what a kernel does besides the sums

// What a part of a row leaves for the kernel that joins them.
struct Part {
  float r, s, u, pad;
};

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
  int64_t rows[P];
  int32_t tile0[P + 1];
  uint32_t block0;
  int32_t N;
  int32_t top;
  float scale;
  uint32_t V;
  uint32_t stride;
  bool through;   // every row of dlogits starts on a line
  int32_t parts;  // of a row, a workgroup each; 1: rows whole
  uint32_t slices;  // of a row in the gradient, a workgroup each
  Part* part;     // [rows of all ranks][parts]
  uint64_t* best; // [rows of all ranks][parts][top] keys of the alternatives
};

__device__ __forceinline__ float exp2_of(float t) { return __builtin_amdgcn_exp2f(t); }  // below 2^-126: 0

// Unit u of a row of n logits, -inf past its end.
template <class In>
__device__ __forceinline__ u32x4 load_logits(const char* row, uint32_t n, uint32_t u) {
  typedef AnyUnit<In> U;
  const uint32_t at = u * U::VE, left = n > at ? min(n - at, static_cast<uint32_t>(U::VE)) : 0;
  return U::load(row + static_cast<uint64_t>(u) * 16, left, 0, In::ES == 2 ? 0xFF80u : 0xFF800000u);
}

// Sums of a set of logits relative to r, which is -kLargest for what is lower: sums of 0 beside any other logit.  Where
// the largest r of a row is that, or kLargest and more, its sums are made again from differences of logits.
struct Stat {
  float r, s, u;
};
constexpr Stat kNothing{-kLargest, 0.0f, 0.0f};

// c's sums relative to r.
__device__ __forceinline__ void raise(Stat& c, float r) {
  const float d = c.r - r, f = exp2_of(d);
  c.u = f * fmaf(c.s, d, c.u);
  c.s *= f;
  c.r = r;
}

// One step of a reduction over a wavefront: lanes read the lane that `ctrl` names, `none` where there is none or
// their row of 16 is not in `rows`.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float x, float none) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(x), CTRL, ROWS, 0xF, false));
}

// Reduces a wavefront's values with f: one, two, four and eight lanes down each row of 16, then row 0 into 1 and 2 into
// 3, then 1 into 2 and 3, and the last lane has it all.  About 60 cycles, a tenth of what exchanges through LDS take.
template <class F>
__device__ __forceinline__ float wave_reduce(float x, float none, F f) {
  x = f(x, dpp<0x111, 0xF>(x, none));
  x = f(x, dpp<0x112, 0xF>(x, none));
  x = f(x, dpp<0x114, 0xF>(x, none));
  x = f(x, dpp<0x118, 0xF>(x, none));
  x = f(x, dpp<0x142, 0xA>(x, none));
  x = f(x, dpp<0x143, 0xC>(x, none));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), kWave - 1));
}

// The largest of a wavefront's values, NaN left out; every lane gets it, as with the rest.
__device__ __forceinline__ float wave_max(float x) {
  return wave_reduce(x, -kInf, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_add(float x) {
  return wave_reduce(x, 0.0f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ Stat wave_stat(Stat c) {
  raise(c, wave_max(c.r));
  return Stat{c.r, wave_add(c.s), wave_add(c.u)};
}

// Keeps the compiler from carrying the widened values of one pass over the registers to the next, at twice their size.
template <int NV>
__device__ __forceinline__ void forget(u32x4 (&x)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) asm volatile("" : "+v"(x[j]));
}

// Sum of VE values in a tree.
template <int VE>
__device__ __forceinline__ float tree(const float (&x)[VE]) {
  if constexpr (VE == 8) return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  else return (x[0] + x[1]) + (x[2] + x[3]);
}

// Adds NV units, those of them that start before unit `units` counted from u0 (the group's first) in steps of LANES, to
// a lane's sums; c2 = scale log2(e).  Returns their maximum (NaN left out); far is set where an x is -inf.  Such an x
// makes 0 * -inf of t 2^t: units where that shows are added again with a limit on t, which is one operation in ten that
// the others save.
template <class In, int LANES, int NV>
__device__ __forceinline__ float add(Stat& c, u32x4 (&x)[NV], uint32_t u0, uint32_t units, float c2, bool& far) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE;
  float m = -kInf;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (u0 + j * LANES >= units) break;
    float v[VE];
    U::widen(x[j], v);
#pragma unroll
    for (int e = 0; e < VE; ++e) m = fmaxf(m, v[e]);
  }
  const float r = m * c2;
  if (r > c.r) raise(c, r);
  const float base = c.r;
  forget(x);
  float s = 0.0f, u = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (u0 + j * LANES >= units) break;
    float v[VE], p[VE];
    U::widen(x[j], v);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      v[e] = fmaf(v[e], c2, -base);
      p[e] = exp2_of(v[e]);
      v[e] *= p[e];
    }
    s += tree<VE>(p);
    float tu = tree<VE>(v);
    if (tu != tu) {
      far = true;
      asm volatile("" : "+v"(x[j]));
      U::widen(x[j], v);
#pragma unroll
      for (int e = 0; e < VE; ++e) v[e] = p[e] * fmaxf(fmaf(v[e], c2, -base), kFarBelow);
      tu = tree<VE>(v);
    }
    u += tu;
  }
  forget(x);
  c.s += s;
  c.u += u;
  return m;
}

// The group's Stat; every lane gets it.  lds: one per wavefront.
template <int LANES>
__device__ __forceinline__ Stat group_stat(Stat c, Stat* lds) {
  c = wave_stat(c);
  if constexpr (LANES > kWave) {
    constexpr int W = LANES / kWave;
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = c;
    __syncthreads();
    c = kNothing;
    if (threadIdx.x % kWave < W) c = lds[threadIdx.x % kWave];
    c = wave_stat(c);
  }
  return c;
}

// The sums of a row whose logits are too large for r, relative to its largest logit m (0 where there is none): t = (x - m)
// scale log2(e), which is exact where it counts.  lds: one per wavefront, from a group_stat.
template <class In, int LANES>
__device__ __forceinline__ Stat sums_from(const char* row, uint32_t V, float c2, Stat* lds, float& m) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE, W = LANES / kWave;
  const uint32_t units = (V + VE - 1) / VE, lane = threadIdx.x % LANES;
  float v[VE];
  m = -kInf;
#pragma unroll 1
  for (uint32_t u = lane; u < units; u += LANES) {
    U::widen(load_logits<In>(row, V, u), v);
#pragma unroll
    for (int e = 0; e < VE; ++e) m = fmaxf(m, v[e]);
  }
  m = wave_max(m);
  if constexpr (W > 1) {
    __syncthreads();
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave].r = m;
    __syncthreads();
    for (int w = 0; w < W; ++w) m = fmaxf(m, lds[w].r);
    __syncthreads();
  }
  Stat c = kNothing;
  if (m == kInf) c.s = m - m;   // NaN
  if (fabsf(m) == kInf) m = 0.0f;
#pragma unroll 1
  for (uint32_t u = lane; u < units; u += LANES) {
    U::widen(load_logits<In>(row, V, u), v);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float t = (v[e] - m) * c2, p = exp2_of(t);
      c.s += p;
      c.u += p * fmaxf(t, kFarBelow);
    }
  }
  return group_stat<LANES>(c, lds);
}

// ------------------------------------------------------------- alternatives
//
// Value v of token id comes before another if it is larger, or equal and of a lower
// id; NaN never counts.  Of every wavefront at least ceil(k / wavefronts) lanes hold
// a value that reaches the threshold the lanes' maxima give, so k values of a tile do,
// and few others: these are listed in LDS, and a value's place is the number of
// listed ones before it.  Where more reach it than the list holds (equal values,
// rows with few tokens left), the tile's k first are found one after the other.

constexpr int kListed = 512;
constexpr int kKept = 128;     // listed values that the next tile starts with at most; with the k first of it they fit

// A value of a token as one number, larger for what comes first; 0 for nothing.  -0 counts as 0.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t id) {
  const uint32_t b = __float_as_uint(v + 0.0f), k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return static_cast<uint64_t>(k) << 32 | ~id;
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t k = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint32_t id_of(uint64_t key) { return ~static_cast<uint32_t>(key); }

struct TopList {
  alignas(16) uint64_t e[kListed];
  int n;       // listed, or more than kListed where some found no room
  float floor; // the threshold that the tiles so far give
};

// A value that at least q lanes' m reach.
__device__ __forceinline__ float qth_largest(float m, int q) {
  float t = kInf;
  for (int i = 0; i < q; ++i) {
    t = wave_max(m);
    const uint64_t at = __ballot(m == t);
    if (at && static_cast<int>(threadIdx.x % kWave) == __ffsll(static_cast<unsigned long long>(at)) - 1) m = -kInf;
  }
  return t;
}

// All lanes of a group have come here, and see each other's LDS.
template <int LANES>
__device__ __forceinline__ void group_sync() {
  if constexpr (LANES > kWave) {
    __syncthreads();
  } else {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Puts the k first of the n listed in order, EACH of them at most per lane.
template <int LANES, int EACH>
__device__ __forceinline__ void order_list(TopList& list, int n, int k) {
  constexpr int AHEAD = 8;
  const int lane = threadIdx.x % LANES;
  uint64_t mine[EACH];
  int place[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    mine[i] = lane + i * LANES < n ? list.e[lane + i * LANES] : 0;
    place[i] = 0;
  }
  for (int j = 0; j < n; j += AHEAD) {
    uint64_t other[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) other[q] = list.e[j + q];   // kListed is a multiple of AHEAD
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (i * LANES >= n) break;
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) place[i] += j + q < n && other[q] > mine[i];
    }
  }
  group_sync<LANES>();
#pragma unroll
  for (int i = 0; i < EACH; ++i)
    if (lane + i * LANES < n && place[i] < k) list.e[place[i]] = mine[i];
}

// Keeps the k first of the listed, in order, and the last of them as the floor.
template <int LANES>
__device__ __forceinline__ void keep_first(TopList& list, int k) {
  const int lane = threadIdx.x % LANES, n = list.n;
  if (n <= LANES) order_list<LANES, 1>(list, n, k);
  else order_list<LANES, (kListed + LANES - 1) / LANES>(list, n, k);
  group_sync<LANES>();
  if (lane == 0) {
    list.n = min(n, k);
    if (n >= k) list.floor = fmaxf(list.floor, value_of(list.e[k - 1]));
  }
  group_sync<LANES>();
}

// The largest of the group's keys; every lane gets it.
template <int LANES>
__device__ __forceinline__ uint64_t group_first(uint64_t x, uint64_t* lds) {
  const auto take = [&](int o) {
    const uint32_t lo = __shfl_xor(static_cast<uint32_t>(x), o), hi = __shfl_xor(static_cast<uint32_t>(x >> 32), o);
    x = max(x, static_cast<uint64_t>(hi) << 32 | lo);
  };
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) take(o);
  if constexpr (LANES > kWave) {
    constexpr int W = LANES / kWave;
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = x;
    __syncthreads();
    x = lds[threadIdx.x % W];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) take(o);
    __syncthreads();
  }
  return x;
}

// Lists what a tile holds of the row's k first.  m: the largest of the lane's values; each(t, f) calls f(v, id) for those
// of them that reach t.
template <int LANES, class Each>
__device__ __forceinline__ void list_tile(TopList& list, int k, float m, float* marks, uint64_t* firsts, Each each) {
  constexpr int W = LANES / kWave;
  float t = qth_largest(m, (k + W - 1) / W);
  if constexpr (W > 1) {
    if (threadIdx.x % kWave == 0) marks[threadIdx.x / kWave] = t;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) t = fminf(t, marks[w]);
  }
  t = fmaxf(t, list.floor);
  const int had = list.n;
  group_sync<LANES>();
  if (m >= t)
    each(t, [&](float v, uint32_t id) {
      const int at = atomicAdd(&list.n, 1);
      if (at < kListed) list.e[at] = key_of(v, id);
    });
  group_sync<LANES>();
  if (list.n > kListed) {
    uint64_t last = ~uint64_t(0);
    for (int i = 0; i < k; ++i) {
      uint64_t b = 0;
      each(-kInf, [&](float v, uint32_t id) {
        const uint64_t key = key_of(v, id);
        if (key < last) b = max(b, key);
      });
      last = group_first<LANES>(b, firsts);
      if (threadIdx.x % LANES == 0) list.e[had + i] = last;
    }
    if (threadIdx.x % LANES == 0) list.n = had + k;
    group_sync<LANES>();
  }
  if (threadIdx.x % LANES == 0) list.floor = t;
  group_sync<LANES>();
}

// The same for a tile of logits, u0 the lane's first unit.
template <class In, int LANES, int NV>
__device__ __forceinline__ void list_logits(TopList& list, int k, u32x4 (&x)[NV], float m, uint32_t u0, uint32_t V, float* marks,
                                            uint64_t* firsts) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE;
  list_tile<LANES>(list, k, m, marks, firsts, [&](float t, auto take) {
    forget(x);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[VE], most = -kInf;
      U::widen(x[j], v);
#pragma unroll
      for (int e = 0; e < VE; ++e) most = fmaxf(most, v[e]);
      if (!(most >= t)) continue;
      uint32_t id = (u0 + j * LANES) * VE;
      asm volatile("" : "+v"(id));   // else the tile's ids are kept in as many registers from one round to the next
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (v[e] >= t && id + e < V) take(v[e], id + e);
    }
  });
}

// ------------------------------------------------------------- gradient

// dx of one logit is -p (a + b t), and `hit` more at the target.  Behind the sums t = x c - r and p = 2^t k: k = 1 / S,
// or 1 for bf16 results, whose r holds log2 S too.  SAVED: from a saved lse, t = x scale - lse and p = e^t: the factor
// log2(e) would round lse before the difference is taken, and 1 - p of a sure target is what that leaves; t above 0 is
// lse's own rounding.  FAR: t may be -inf, or its product with b beyond all numbers, where p is 0; and t = (x - m) c - r.
struct RowGrad {
  float m, c, r, k, a, b, hit;
  uint32_t target;   // ~0: none
  float none;        // dx where p is 0, if a or b is so large, or no number, that a limit on t does not give it
  // p (a + b t) is 0 where p is, for every finite t.
  __device__ __forceinline__ bool any_t() const { return fabsf(b) < 0.25f && fabsf(a) < kLargeFactor; }
  // And for every t down to kNoneBelow.
  __device__ __forceinline__ bool limited_t() const { return fabsf(b) < kLargeFactor && fabsf(a) < kLargeFactor; }
};

// dx of what has probability 0: 0, or NaN where a factor is no finite number.
__device__ __forceinline__ float none_of(bool empty, float dlp, float dent) { return empty ? 0.0f : 0.0f * dlp + 0.0f * dent; }

// Gradients of unit u from its logits, stored; zeros in columns V .. stride - 1.
template <class In, bool SAVED, bool FAR>
__device__ __forceinline__ void put_grads(const RowGrad& g, const u32x4& x, char* out, uint32_t u, uint32_t V, uint32_t stride,
                                          bool through) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE;
  const uint32_t at = u * VE;
  if (at >= stride) return;
  float v[VE];
  U::widen(x, v);
  float t;
  const auto p_of = [&](float x) {   // and its t
    t = fmaf(FAR && !SAVED ? x - g.m : x, g.c, -g.r);
    if (SAVED) t = t > 0.0f ? 0.0f : t;
    const float p = exp2_of(SAVED ? t * kLog2E : t);
    return !SAVED && In::ES == 4 ? p * g.k : p;   // bf16: r holds log2 S
  };
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const float p = p_of(v[e]);
    v[e] = -p * fmaf(g.b, FAR ? fmaxf(t, kNoneBelow) : t, g.a);
  }
  if (FAR && __builtin_amdgcn_readfirstlane(!g.limited_t())) {
    u32x4 again = x;
    asm volatile("" : "+v"(again));   // or the values would stay in registers for this
    float w[VE];
    U::widen(again, w);
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (p_of(w[e]) == 0.0f) v[e] = g.none;
  }
  if (g.target - at < VE)
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (g.target == at + e) v[e] += g.hit;
  if (at + VE > V)
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (at + e >= V) v[e] = 0.0f;
  U::store(out + static_cast<uint64_t>(u) * 16, min(stride - at, static_cast<uint32_t>(VE)), 0, U::narrow(v), through);
}

// The row's target, ~0 for none.
template <int P>
__device__ __forceinline__ uint32_t target_of(const LogprobArgs<P>& a, int rank, int64_t r) {
  const uint32_t t = a.targets[rank] ? static_cast<uint32_t>(a.targets[rank][r]) : ~0u;
  return t < a.V ? t : ~0u;
}

// ------------------------------------------------------------- kernels

// Row of this group, or false past the rank's last.
template <int LANES, int P>
__device__ __forceinline__ bool row_of(const LogprobArgs<P>& a, int32_t block, int& rank, int64_t& r) {
  rank = rank_of<P>(a.tile0, a.N, block);
  constexpr int GROUPS = LANES == kWave ? kThreads / kWave : 1;
  r = static_cast<int64_t>(block - a.tile0[rank]) * GROUPS + (GROUPS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) : 0);
  return r < a.rows[rank];
}

// A row's numbers from its sums.
struct RowSums {
  float c2, m = 0.0f, base, log2_s, inv_s, entropy, lse;
  bool large, empty;   // large: sums relative to the logit m
  // c: the sums of the group's lanes; again(m) makes them anew from the row's logits.
  template <class Again>
  __device__ __forceinline__ RowSums(Stat c, float scale, Again again) : c2(scale * kLog2E), large(!(fabsf(c.r) < kLargest)) {
    if (large) c = again(c2, m);
    empty = c.s == 0.0f;
    base = large ? 0.0f : c.r;
    log2_s = empty ? 0.0f : __log2f(c.s);
    inv_s = empty ? 0.0f : 1.0f / c.s;
    entropy = empty ? 0.0f : kLn2 * (log2_s - c.u * inv_s);
    lse = empty ? -kInf : fmaf(scale, m, kLn2 * (base + log2_s));
  }
  __device__ __forceinline__ float log_p(float x) const { return empty ? -kInf : kLn2 * (fmaf(x - m, c2, -base) - log2_s); }
};

// Stores a row's numbers (from one lane); target ~0: none, else its logit is given.
template <int P>
__device__ __forceinline__ void put_row(const LogprobArgs<P>& a, int rank, int64_t r, const RowSums& n, uint32_t target, float given) {
  if (a.lse[rank]) a.lse[rank][r] = n.lse;
  if (a.entropy[rank]) a.entropy[rank][r] = n.entropy;
  if (a.logprob[rank]) a.logprob[rank][r] = target == ~0u ? 0.0f : n.log_p(given);
}

// Stores the alternatives, one per lane.
template <int LANES, int P>
__device__ __forceinline__ void put_top(const LogprobArgs<P>& a, int rank, int64_t r, const RowSums& n, TopList& list) {
  keep_first<LANES>(list, a.top);
  const int lane = threadIdx.x % LANES;
  if (lane < a.top) {
    const bool some = lane < list.n;
    a.top_ids[rank][r * a.top + lane] = some ? static_cast<int32_t>(id_of(list.e[lane])) : -1;
    a.top_logprob[rank][r * a.top + lane] = n.log_p(some ? value_of(list.e[lane]) : -kInf);
  }
}

template <class In, int LANES, int NV, int MODE, bool SPLIT, int P>
__global__ void __launch_bounds__(LANES == kWave ? kThreads : LANES) logprob_kernel(const LogprobArgs<P> a) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE, W = LANES / kWave;
  __shared__ Stat stats[W];
  __shared__ float marks[MODE == kTop ? W : 1];
  __shared__ uint64_t firsts[MODE == kTop ? W : 1];
  __shared__ TopList lists[MODE != kTop ? 1 : LANES == kWave ? kThreads / kWave : 1];
  int rank;
  int64_t r;
  const int32_t block = a.block0 + blockIdx.x;
  if (!row_of<LANES, P>(a, SPLIT ? block / a.parts : block, rank, r)) return;
  const int lane = threadIdx.x % LANES;
  const uint64_t off = static_cast<uint64_t>(r) * a.stride * In::ES;
  const char* row = a.logits[rank] + off;
  const uint32_t all = (a.V + VE - 1) / VE, share = SPLIT ? (all + a.parts - 1) / a.parts : all;
  const uint32_t first = SPLIT ? min(block % a.parts * share, all) : 0, units = min(first + share, all);
  const float c2 = a.scale * kLog2E;
  const uint32_t target = SPLIT ? ~0u : target_of(a, rank, r);
  const float dlp = MODE == kGrad && target != ~0u ? a.dlogprob[rank][r] : 0.0f;
  const float dent = MODE == kGrad && a.dentropy[rank] ? a.dentropy[rank][r] : 0.0f;
  Stat c = kNothing;
  TopList& list = lists[MODE == kTop && LANES == kWave ? threadIdx.x / kWave : 0];
  if constexpr (MODE == kTop) {
    if (lane == 0) {
      list.n = 0;
      list.floor = -kInf;
    }
    group_sync<LANES>();
  }
  u32x4 x[NV];
  const uint32_t V = SPLIT ? min(a.V, units * VE) : a.V;             // the logits from there on are the next part's
  const auto fetch = [&](uint32_t u0) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      x[j] = u0 - lane + j * LANES < units ? load_logits<In>(row, V, u0 + j * LANES) : u32x4{0, 0, 0, 0};
  };
  bool far = false;
  float given = 0.0f;
  for (uint32_t u0 = first + lane; u0 - lane < units; u0 += NV * LANES) {
    if constexpr (MODE == kTop)
      if (list.n > kKept) keep_first<LANES>(list, a.top);            // for a higher floor
    fetch(u0);
    if (u0 - lane == first && target != ~0u) given = In::one(row, target);   // before dlogits may overwrite it
    const float m = add<In, LANES, NV>(c, x, u0 - lane, units, c2, far);
    if constexpr (MODE == kTop) list_logits<In, LANES, NV>(list, a.top, x, m, u0, V, marks, firsts);
  }
  c = group_stat<LANES>(c, stats);
  if constexpr (SPLIT) {
    uint64_t at = block;                                             // rows of all ranks are numbered as their parts are
    if (lane == 0) a.part[at] = Part{c.r, c.s, c.u, 0.0f};
    if constexpr (MODE == kTop) {
      keep_first<LANES>(list, a.top);
      if (lane < a.top) a.best[at * a.top + lane] = lane < list.n ? list.e[lane] : 0;
    }
    return;
  }
  const RowSums n(c, a.scale, [&](float c2, float& m) { return sums_from<In, LANES>(row, a.V, c2, stats, m); });
  if (lane == 0) put_row(a, rank, r, n, target, given);
  if constexpr (MODE == kTop) put_top<LANES>(a, rank, r, n, list);
  if constexpr (MODE == kGrad) {
    const float hit = n.empty ? 0.0f : a.scale * dlp;
    // dlogprob p + dentropy p (log p + entropy), log p = ln2 t or ln2 (t - log2 S)
    const float b = a.scale * dent * kLn2, norm = In::ES == 2 ? n.log2_s : 0.0f;
    const RowGrad g{n.m, c2, n.base + norm, n.inv_s, hit + a.scale * dent * n.entropy - b * (n.log2_s - norm), b, hit,
                    target, none_of(n.empty, dlp, dent)};
    char* out = a.dlogits[rank] + off;
    const uint32_t wide = (a.stride + VE - 1) / VE;
    // a wavefront takes the limits on t where one of its lanes met a -inf, and where b t of a finite t may be beyond all
    // numbers (8 x 4096 rows of 32000 bf16: 766 us with them, 751 without); columns past V are filled with -inf
    const bool limits = __any(far) || n.large || a.V < wide * VE || !g.any_t();
    for (uint32_t u1 = lane; u1 - lane < wide; u1 += NV * LANES) {
      if (wide > NV * LANES)
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = load_logits<In>(row, a.V, u1 + j * LANES);
      if (limits) {
#pragma unroll
        for (int j = 0; j < NV; ++j) put_grads<In, false, true>(g, x[j], out, u1 + j * LANES, a.V, a.stride, a.through);
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) put_grads<In, false, false>(g, x[j], out, u1 + j * LANES, a.V, a.stride, a.through);
      }
    }
  }
}

// Joins the parts of a row, at most kWave of them.
template <class In, bool TOP, int P>
__global__ void __launch_bounds__(kThreads) logprob_join_kernel(const LogprobArgs<P> a) {
  __shared__ Stat stats[kThreads / kWave];
  __shared__ float marks[kThreads / kWave];
  __shared__ uint64_t firsts[kThreads / kWave];
  __shared__ TopList list;
  int rank;
  int64_t r;
  const int32_t block = a.block0 + blockIdx.x;
  row_of<kThreads, P>(a, block, rank, r);
  const uint32_t target = target_of(a, rank, r);
  Stat c = kNothing;
  const int lane = threadIdx.x % kWave;
  if (lane < a.parts) {
    const Part p = a.part[static_cast<uint64_t>(block) * a.parts + lane];
    c = Stat{p.r, p.s, p.u};
  }
  c = group_stat<kWave>(c, nullptr);
  const char* row = a.logits[rank] + static_cast<uint64_t>(r) * a.stride * In::ES;
  const RowSums n(c, a.scale, [&](float c2, float& m) { return sums_from<In, kThreads>(row, a.V, c2, stats, m); });
  if (threadIdx.x == 0) put_row(a, rank, r, n, target, target == ~0u ? 0.0f : In::one(row, target));
  if constexpr (TOP) {
    constexpr int EACH = kMostParts * kWave / kThreads;
    const int count = a.parts * a.top;
    const uint64_t* best = a.best + static_cast<uint64_t>(block) * count;
    uint64_t x[EACH];
    float m = -kInf;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int i = threadIdx.x + j * kThreads;
      x[j] = i < count ? best[i] : 0;
      if (x[j]) m = fmaxf(m, value_of(x[j]));
    }
    if (threadIdx.x == 0) {
      list.n = 0;
      list.floor = -kInf;
    }
    __syncthreads();
    list_tile<kThreads>(list, a.top, m, marks, firsts, [&](float t, auto take) {
#pragma unroll
      for (int j = 0; j < EACH; ++j)
        if (x[j] && value_of(x[j]) >= t) take(value_of(x[j]), id_of(x[j]));
    });
    put_top<kThreads>(a, rank, r, n, list);
  }
}

// The gradient from the saved lse and entropy, kSlice units of a row per lane group: workgroups that run side by side
// then read and write memory side by side (2 x 1024 x 131072 bf16: 178 us, 212 with a workgroup per row; 8 x 4096 x 32000
// 786 and 803).
constexpr int kSlice = 4;   // units per lane

template <class In, int LANES, int P>
__global__ void __launch_bounds__(kThreads) logprob_backward_kernel(const LogprobArgs<P> a) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE;
  int rank;
  int64_t r;
  const uint64_t block = a.block0 + static_cast<uint64_t>(blockIdx.x);
  const uint32_t line = static_cast<uint32_t>(block / a.slices), slice = static_cast<uint32_t>(block - static_cast<uint64_t>(line) * a.slices);
  if (!row_of<LANES, P>(a, static_cast<int32_t>(line), rank, r)) return;
  const int lane = threadIdx.x % LANES;
  const uint32_t target = target_of(a, rank, r);
  const float lse = a.lse[rank][r];
  const float dlp = a.dlogprob[rank][r], dent = a.dentropy[rank] ? a.dentropy[rank][r] : 0.0f;
  const float entropy = a.entropy[rank] ? a.entropy[rank][r] : 0.0f;
  const uint64_t off = static_cast<uint64_t>(r) * a.stride * In::ES;
  const uint32_t u0 = slice * (kSlice * LANES) + lane;
  u32x4 x[kSlice];
#pragma unroll
  for (int j = 0; j < kSlice; ++j) x[j] = load_logits<In>(a.logits[rank] + off, a.V, u0 + j * LANES);
  const bool empty = lse == -kInf;
  const float hit = target == ~0u || empty ? 0.0f : a.scale * dlp;
  const RowGrad g{0.0f, a.scale, empty ? 0.0f : lse, 1.0f, hit + a.scale * dent * entropy, a.scale * dent, hit, target,
                  none_of(empty, target == ~0u ? 0.0f : dlp, dent)};
#pragma unroll
  for (int j = 0; j < kSlice; ++j) put_grads<In, true, true>(g, x[j], a.dlogits[rank] + off, u0 + j * LANES, a.V, a.stride, a.through);
}

// ------------------------------------------------------------- host side

template <class In, int MODE, int LANES, int NV, int P>
gc_status launch_rows(LogprobArgs<P>& a, const gci::LogprobCall& c) {
  constexpr int threads = LANES == kWave ? kThreads : LANES;
  fill_blocks<P>(a.tile0, c.tokens, c.nranks, threads / LANES);
  return launch_blocks(logprob_kernel<In, LANES, NV, MODE, false, P>, a, a.tile0[c.nranks], threads, c.stream);
}

// Lanes of a row and their units.  A wavefront holds a short row: 8 x 16384 rows of 1000 bf16 take 73 us for the sums
// and 121 with the gradient so, 192 and 277 with 256 lanes (of 2000, the longest: 108 and 218, 196 and 332).  A longer
// row's gradient wants all of it in registers, in few lanes: of 8192 183 us with 256 lanes of 4 units, 215 with 512; of
// 16384 368 with 512 of 4, 398 of 8; of 32000 728 with 512 of 8, 759 with 256 of 16, 775 with 1024 of 4 (8 x 4096 rows).
// Beyond what registers hold tiles of 4 units cost less at the row's end than those of 8: of 69632 264 us and 299, of
// 131072 273 and 274 (7 x 550 and 2 x 1024 rows), 300 and 292 with 512 of 4, 314 and 297 with 256 of 4.  Sums alone
// stream: 316 us with 256 lanes of 4, 314 of 8, 335 with 512 of 8, 366 with 1024 of 4; with five alternatives 256 of 8
// take 108 us, of 4 126, 512 of 4 144 (4 x 2048 rows).  Where rows are too few to fill the chip, more lanes finish one
// sooner: 64 rows of 32003 fp32 5.3 us with 1024 lanes, 9.7 with 256, with five alternatives 12.7 and 19.3.
// More than 8 ranks have one form, chosen for the size of the library and not by time: 64 x 2048 rows of 1000 take 906
// us and with the gradient 1075, as 8 x 16384 76 and 127; 64 x 512 of 32000 387 and 777, as 8 x 4096 325 and 729.
template <class In, int MODE, int P>
gc_status launch_mode(LogprobArgs<P>& a, const gci::LogprobCall& c) {
  if constexpr (P > 8) {
    return launch_rows<In, MODE, 512, 8, P>(a, c);   // one form for the many ranks
  } else {
    const uint64_t units = ((MODE == kGrad ? c.stride : c.vocab) + In::VE - 1) / In::VE;
    if (units <= 4 * kWave) return launch_rows<In, MODE, kWave, 4, P>(a, c);
    if constexpr (MODE == kGrad) {
      if (units <= 4 * 256) return launch_rows<In, MODE, 256, 4, P>(a, c);
      if (units <= 4 * 512) return launch_rows<In, MODE, 512, 4, P>(a, c);
      if (units <= 8 * 512) return launch_rows<In, MODE, 512, 8, P>(a, c);
      return units <= 8 * 1024 ? launch_rows<In, MODE, 1024, 8, P>(a, c) : launch_rows<In, MODE, 1024, 4, P>(a, c);
    } else {
      int64_t rows = 0;
      for (int s = 0; s < c.nranks; ++s) rows += c.tokens[s];
      if (rows < 512 && units > 2 * 1024) return launch_rows<In, MODE, 1024, 8, P>(a, c);
      return launch_rows<In, MODE, 256, MODE == kTop ? 8 : 4, P>(a, c);
    }
  }
}

// Few rows: a workgroup per part, and one per row that joins them (one row of 131072 bf16 with 20 alternatives: 13 us, 25
// by one workgroup).
template <class In, int P>
gc_status launch_parts(LogprobArgs<P>& a, const gci::LogprobCall& c) {
  fill_blocks<P>(a.tile0, c.tokens, c.nranks, 1);
  const int32_t rows = a.tile0[c.nranks];
  a.part = static_cast<Part*>(c.scratch);
  a.best = reinterpret_cast<uint64_t*>(a.part + static_cast<uint64_t>(rows) * a.parts);
  const gc_status st = c.top ? launch_blocks(logprob_kernel<In, 256, 4, kTop, true, P>, a, rows * a.parts, 256, c.stream)
                             : launch_blocks(logprob_kernel<In, 256, 4, kStats, true, P>, a, rows * a.parts, 256, c.stream);
  if (st != GC_OK) return st;
  return c.top ? launch_blocks(logprob_join_kernel<In, true, P>, a, rows, kThreads, c.stream)
               : launch_blocks(logprob_join_kernel<In, false, P>, a, rows, kThreads, c.stream);
}

template <class In, int P>
gc_status backward_rows(LogprobArgs<P>& a, const gci::LogprobCall& c) {
  const uint64_t units = (c.stride + In::VE - 1) / In::VE;
  const bool wave = units <= kSlice * kWave;   // a wavefront holds a row
  fill_blocks<P>(a.tile0, c.tokens, c.nranks, wave ? kThreads / kWave : 1);
  a.slices = wave ? 1 : static_cast<uint32_t>((units + kSlice * kThreads - 1) / (kSlice * kThreads));
  const uint64_t blocks = static_cast<uint64_t>(a.tile0[c.nranks]) * a.slices;
  return wave ? launch_blocks(logprob_backward_kernel<In, kWave, P>, a, blocks, kThreads, c.stream)
              : launch_blocks(logprob_backward_kernel<In, kThreads, P>, a, blocks, kThreads, c.stream);
}

template <class In, int P>
gc_status logprob_typed(const gci::LogprobCall& c, bool backward) {
  LogprobArgs<P> a{};
  uint64_t m = c.stride * In::ES;
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
    if (c.dlogits && c.tokens[s]) m |= reinterpret_cast<uint64_t>(c.dlogits[s]);
    a.rows[s] = c.tokens[s];
  }
  a.N = c.nranks;
  a.top = c.top;
  a.scale = c.scale;
  a.V = static_cast<uint32_t>(c.vocab);
  a.stride = static_cast<uint32_t>(c.stride);
  a.through = m % kLine == 0;
  if (backward) return backward_rows<In, P>(a, c);
  a.parts = c.dlogits ? 1 : c.parts;
  if (a.parts > 1) return launch_parts<In, P>(a, c);
  if (c.top) return launch_mode<In, kTop, P>(a, c);
  return c.dlogits ? launch_mode<In, kGrad, P>(a, c) : launch_mode<In, kStats, P>(a, c);
}

gc_status logprob_any(const gci::LogprobCall& c, bool backward) {
  if (c.t == GC_BF16) return c.nranks <= 8 ? logprob_typed<InBf16, 8>(c, backward) : logprob_typed<InBf16, 64>(c, backward);
  return c.nranks <= 8 ? logprob_typed<InF32, 8>(c, backward) : logprob_typed<InF32, 64>(c, backward);
}

}  // namespace

namespace gci {

gc_status launch_token_logprob_backward(const LogprobCall& c) { return logprob_any(c, true); }

gc_status launch_token_logprob(const LogprobCall& c) {
  if (!c.top || !c.dlogits) return logprob_any(c, false);
  // both at once are rare: the alternatives first, then the pass with the gradient, which may overwrite the logits
  LogprobCall part = c;
  part.dlogits = nullptr;
  const gc_status st = logprob_any(part, false);
  if (st != GC_OK) return st;
  part = c;
  part.top = 0;
  return logprob_any(part, false);
}

}  // namespace gci
