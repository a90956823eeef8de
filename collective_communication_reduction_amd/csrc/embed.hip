// Token embedding and its gradient, for gfx950.
//
//   out[t] = scale * W[id t]          dW[v] = scale * sum over t with id t = v of dout[t]
//
// The gradient first sorts the tokens by id, stably (counting sort by one or two
// digits of the id), so that each row's terms are added in token order whatever
// the timing: results repeat bit for bit, and no atomic touches a gradient.
//
// HBM bytes bound both.  8 x 16384 rows of 4096 bf16 from a vocabulary of 32000: the lookup takes 242 us (1.07 GB written,
// of the weight only what occurs read: 5.5 TB/s; 227 to 261 by the card and by where the frequent rows lie), the gradient 566 (561 to
// 596): sums and cleared rows 537 to 558 (3.17 GB read and written, 5.7 to 5.9 TB/s), sort 23, long rows 10.

#include <algorithm>
#include <type_traits>

#include "units.h"

namespace {

using namespace gcdev;

// ------------------------------------------------------------- lookup
//
// Up to a wavefront of lanes share a row's slice, each with up to four units in flight: 8 x 16384 rows of 4096 bf16
// that repeat take 227 us so, 337 with one unit a lane and eight slices, 279 with eight units a lane (distinct rows 385, 388
// and 401).  The weight may stay in the caches, frequent tokens being read again: 227 us, 271 with streaming loads.

template <int P>
struct EmbeddingArgs {
  const char* w[P];
  const int32_t* ids[P];
  char* out[P];
  int64_t tok[P];
  int32_t tile0[P + 1];
  uint32_t block0;
  int32_t N;
  uint32_t vocab;
  uint64_t H;
  uint64_t units;       // per row
  uint32_t slices;      // of a row, NV << lanes_log2 units each
  int32_t lanes_log2;   // lanes that share a row's slice
  bool through;         // every row written starts on a line
  float scale;
};

template <class In, int NV, int P>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const EmbeddingArgs<P> a) {
  typedef AnyUnit<In> U;
  constexpr int VE = U::VE;
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const uint64_t q = (static_cast<uint64_t>(block - a.tile0[rank]) * kThreads + threadIdx.x) >> a.lanes_log2;
  const uint64_t row = a.slices == 1 ? q : q / a.slices;
  if (row >= static_cast<uint64_t>(a.tok[rank])) return;
  const uint32_t lanes = 1u << a.lanes_log2;
  const uint32_t u0 = static_cast<uint32_t>((q - row * a.slices) * (static_cast<uint64_t>(NV) << a.lanes_log2)) + (threadIdx.x & (lanes - 1));
  const uint32_t id = static_cast<uint32_t>(a.ids[rank][row]);
  const bool known = id < a.vocab;
  char* dst = a.out[rank] + row * a.H * In::ES;
  const char* src = a.w[rank] + static_cast<uint64_t>(known ? id : 0) * a.H * In::ES;
  const uint32_t H = static_cast<uint32_t>(a.H);
  u32x4 x[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    x[j] = known && u0 + j * lanes < a.units ? U::template load<true>(src, H, U::start(H, u0 + j * lanes)) : u32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (u0 + j * lanes >= a.units) continue;
    float v[VE];
    U::widen(x[j], v);
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = known ? v[e] * a.scale : 0.0f;
    U::store(dst, H, U::start(H, u0 + j * lanes), U::narrow(v), a.through);
  }
}

// ------------------------------------------------------------- sort by token
//
// Bounded by its launches and their latency, 5 to 7 us each for 8 x 16384 tokens: counts per piece of 1024 tokens and
// places from the counts of all pieces, once per digit of up to 11 bits (two cover any vocabulary taken here, and the
// eight wavefronts' counts fill 64 KB of LDS).  Inside a wavefront entries of the same digit find each other by
// ballots, so that their order is kept.

constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kSortRun = (1 << gci::kEmbeddingDigit) / kSortThreads;   // digits per thread

template <int P>
struct SortArgs {
  const int32_t* ids[P];
  int64_t tok[P];
  int64_t at[P];          // first entry of each rank in the scratch lists
  int32_t tile0[P + 1];
  uint32_t block0;
  int32_t N;
  int32_t chunk;          // entries per workgroup
  uint32_t vocab;
  int32_t low_bits;       // of the first pass's digit
  int32_t high_bits;      // of the second's, 0: one pass
  uint64_t* pairs;        // id << 32 | token, between the passes
  int32_t* keys;          // sorted ids and their tokens
  int32_t* perm;
  uint32_t* counts;       // [chunks][1 << bits]
  int32_t* valid;         // tokens of each rank inside the vocabulary
  uint8_t* present;       // [ranks][present_row] whether a token occurs
  uint32_t present_row;   // bytes, a multiple of 16
  int32_t* long_rows;     // count, then the runs where rows of many runs begin
};

// Entry i of the pass's input as id << 32 | token; ~0 for a token outside the vocabulary.
template <bool FIRST, int P>
__device__ __forceinline__ uint64_t sort_entry(const SortArgs<P>& a, int rank, int64_t i, int64_t n) {
  if (i >= n) return ~uint64_t(0);
  if constexpr (FIRST) {
    const uint32_t id = static_cast<uint32_t>(a.ids[rank][i]);
    return id < a.vocab ? static_cast<uint64_t>(id) << 32 | static_cast<uint32_t>(i) : ~uint64_t(0);
  } else {
    return a.pairs[a.at[rank] + i];
  }
}

// A digit of the id: `bits` bits from bit `shift` on.
struct Digit {
  int32_t shift, bits;
  __device__ __forceinline__ uint32_t of(uint64_t entry) const {
    return static_cast<uint32_t>(entry >> (32 + shift)) & ((1u << bits) - 1);
  }
};

// Clears part `mine` of `parts` of the rank's map of tokens, and the count of long rows.
template <int P>
__device__ __forceinline__ void clear_marks(const SortArgs<P>& a, int rank, uint32_t mine, uint32_t parts) {
  u32x4* map = reinterpret_cast<u32x4*>(a.present + static_cast<uint64_t>(rank) * a.present_row);
  for (uint32_t v = mine * kSortThreads + threadIdx.x; v < a.present_row / 16; v += parts * kSortThreads) map[v] = u32x4{0, 0, 0, 0};
  if (rank == 0 && mine == 0 && threadIdx.x == 0) a.long_rows[0] = 0;
}

// Digit counts of one chunk.
template <bool FIRST, int P>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs<P> a) {
  extern __shared__ uint32_t hist[];
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int64_t n = FIRST ? a.tok[rank] : a.valid[rank];
  const int64_t first = static_cast<int64_t>(block - a.tile0[rank]) * a.chunk;
  const Digit digit = FIRST ? Digit{0, a.low_bits} : Digit{a.low_bits, a.high_bits};
  const int bins = 1 << digit.bits;
  if constexpr (FIRST) clear_marks(a, rank, block - a.tile0[rank], a.tile0[rank + 1] - a.tile0[rank]);
  for (int d = threadIdx.x; d < bins; d += kSortThreads) hist[d] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.chunk; i += kSortThreads) {
    const uint64_t e = sort_entry<FIRST>(a, rank, first + i, n);
    if (e != ~uint64_t(0)) atomicAdd(&hist[digit.of(e)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) a.counts[static_cast<uint64_t>(block) * bins + d] = hist[d];
}

// Exclusive sum over the workgroup's threads.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t x, uint32_t* lds, uint32_t& total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  uint32_t s = x;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint32_t t = __shfl_up(s, o);
    if (lane >= o) s += t;
  }
  if (lane == kWave - 1) lds[wave] = s;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    before += w < wave ? lds[w] : 0;
    total += lds[w];
  }
  __syncthreads();
  return before + s - x;
}

// Places chunk `mine` of the rank's n entries: behind all entries of smaller digits,
// those of the same digit in earlier chunks, and those of earlier wavefronts and
// lanes.  ALONE: the rank has this chunk only, whose counts need not be looked up.
// Returns the number of entries of all chunks.
template <bool FIRST, bool LAST, bool ALONE, int P>
__device__ __forceinline__ uint32_t place_chunk(const SortArgs<P>& a, int rank, int64_t n, int32_t mine, int32_t chunks,
                                                uint32_t* next, uint32_t* sums) {
  const Digit digit = FIRST ? Digit{0, a.low_bits} : Digit{a.low_bits, a.high_bits};
  const int bins = 1 << digit.bits, wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int per = a.chunk / kSortWaves;
  const int64_t first = static_cast<int64_t>(mine) * a.chunk + wave * per;
  uint32_t* my = next + wave * bins;   // [wavefront][digit]: entries counted, then the place of the next one
  for (int d = threadIdx.x; d < kSortWaves * bins; d += kSortThreads) next[d] = 0;
  __syncthreads();
  for (int i = lane; i < per; i += kWave) {
    const uint64_t e = sort_entry<FIRST>(a, rank, first + i, n);
    if (e != ~uint64_t(0)) atomicAdd(&my[digit.of(e)], 1u);
  }
  __syncthreads();
  // digits in order, up to four of them per thread: entries of all chunks, and of those before this one
  const int run = (bins + kSortThreads - 1) / kSortThreads;
  const uint32_t* counts = ALONE ? nullptr : a.counts + static_cast<uint64_t>(a.tile0[rank]) * bins;
  const int d0 = threadIdx.x * run;
  uint32_t all[kSortRun] = {}, before[kSortRun] = {}, sum = 0;
#pragma unroll
  for (int k = 0; k < kSortRun; ++k) {
    if (k >= run || d0 + k >= bins) break;
    if constexpr (ALONE) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) all[k] += next[w * bins + d0 + k];
    } else {
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const uint32_t t = counts[static_cast<uint64_t>(c) * bins + d0 + k];
        all[k] += t;
        before[k] += c < mine ? t : 0;
      }
    }
    sum += all[k];
  }
  uint32_t total;
  uint32_t at = block_exclusive(sum, sums, total);
#pragma unroll
  for (int k = 0; k < kSortRun; ++k) {
    const int d = d0 + k;
    if (k >= run || d >= bins) break;
    uint32_t place = at + before[k];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t t = next[w * bins + d];
      next[w * bins + d] = place;
      place += t;
    }
    at += all[k];
  }
  __syncthreads();
  for (int i = 0; i < per; i += kWave) {
    const uint64_t e = sort_entry<FIRST>(a, rank, first + i + lane, i + lane < per ? n : 0);
    const bool ok = e != ~uint64_t(0);
    const uint32_t d = ok ? digit.of(e) : 0;
    uint64_t peers = __ballot(ok);
    for (int b = 0; b < digit.bits; ++b) {
      const uint64_t ones = __ballot(d >> b & 1);
      peers &= d >> b & 1 ? ones : ~ones;
    }
    const int ahead = __popcll(peers & ((uint64_t(1) << lane) - 1));
    const uint32_t place = ok ? my[d] + ahead : 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (ok && ahead == 0) my[d] += __popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (ok) {
      if constexpr (FIRST) a.present[static_cast<uint64_t>(rank) * a.present_row + (e >> 32)] = 1;
      if constexpr (LAST) {
        a.keys[a.at[rank] + place] = static_cast<int32_t>(e >> 32);
        a.perm[a.at[rank] + place] = static_cast<int32_t>(e);
      } else {
        a.pairs[a.at[rank] + place] = e;
      }
    }
  }
  return total;
}

template <bool FIRST, bool LAST, int P>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortArgs<P> a) {
  extern __shared__ uint32_t next[];
  __shared__ uint32_t sums[kSortWaves];
  const int32_t block = a.block0 + blockIdx.x;
  const int rank = rank_of<P>(a.tile0, a.N, block);
  const int32_t mine = block - a.tile0[rank];
  const uint32_t total = place_chunk<FIRST, LAST, false>(a, rank, FIRST ? a.tok[rank] : a.valid[rank], mine,
                                                         a.tile0[rank + 1] - a.tile0[rank], next, sums);
  if (FIRST && mine == 0 && threadIdx.x == 0) a.valid[rank] = static_cast<int32_t>(total);
}

// The whole sort of ranks of few tokens, one workgroup each.
template <int P>
__global__ void __launch_bounds__(kSortThreads) sort_alone_kernel(const SortArgs<P> a) {
  extern __shared__ uint32_t next[];
  __shared__ uint32_t sums[kSortWaves];
  const int rank = blockIdx.x;
  clear_marks(a, rank, 0, 1);
  __threadfence_block();
  __syncthreads();
  uint32_t n;
  if (a.high_bits == 0) {
    n = place_chunk<true, true, true>(a, rank, a.tok[rank], 0, 1, next, sums);
  } else {
    n = place_chunk<true, false, true>(a, rank, a.tok[rank], 0, 1, next, sums);
    __threadfence_block();
    __syncthreads();
    place_chunk<false, true, true>(a, rank, n, 0, 1, next, sums);
  }
  if (threadIdx.x == 0) a.valid[rank] = static_cast<int32_t>(n);
}

// ------------------------------------------------------------- sums of sorted rows
//
// The sorted tokens are cut into runs of equal length, whatever rows they belong
// to, so that frequent tokens spread over the chip.  The run where a row begins
// also takes what the next run holds of it, if the row ends there.  Longer rows
// are left as partial sums, the first of them the tail of the run where the row
// begins, the others the heads of the runs behind, and a second launch adds them up.
// (A group of lanes per row of the vocabulary instead, 8 x 16384 x 4096: 4945 us,
// nearly all of it the most frequent token's.)

constexpr int kClearAhead = 4;   // rows that are looked up together before the empty ones are cleared

template <int P>
struct RowSumArgs {
  const char* dout[P];
  char* dw[P];
  int64_t at[P];
  int32_t run0[P + 1];   // first run of each rank
  uint32_t block0;
  int32_t N;
  uint32_t vocab;
  uint64_t H;
  uint64_t units;        // per row
  uint64_t pitch;        // floats of a partial row
  uint64_t sum_blocks;   // workgroups of the runs; those behind clear rows
  uint32_t slices;       // of a row, NV << lanes_log2 units each
  int32_t lanes_log2;
  bool through;          // every row written starts on a line
  uint32_t clear_rows;   // rows per clearing workgroup
  const int32_t* keys;
  const int32_t* perm;
  const int32_t* valid;
  const uint8_t* present;
  uint32_t present_row;
  int32_t* long_rows;    // count, then the runs where rows of many runs begin
  float* partial;        // [runs][head, tail][pitch]
  int32_t run;           // sorted tokens per run
  float scale;
  bool accumulate;
};

// First of the sorted entries lo .. hi - 1 whose id is above key (hi: none).
__device__ __forceinline__ int past(const int2* entries, int lo, int hi, int32_t key) {
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (entries[mid].x <= key) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// VE sums times scale to a row of n elements: those from element `off` of its unit u (of UNIT elements) on.  With `add`
// they go on top of what is there, each element from one lane alone: what the row's last unit shares with the one before,
// which may be more than the first of its pieces, is left to that.
template <class OutT, int VE, int UNIT>
__device__ __forceinline__ void put_sums(char* row, uint32_t n, uint32_t u, uint32_t off, const float (&acc)[VE], float scale,
                                         bool add, bool through) {
  typedef AnyUnit<OutT, VE> W;
  const uint32_t s = gci::unit_start(n, UNIT, u) + off, here = gci::unit_held(n, UNIT, off, VE);
  char* p = row + static_cast<uint64_t>(s) * OutT::ES;
  float v[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) v[e] = acc[e] * scale;
  if (!add) {
    W::store(p, here, 0, W::narrow(v), through);
    return;
  }
  float old[VE];
  W::widen(W::load(p, here, 0), old);
#pragma unroll
  for (int e = 0; e < VE; ++e) v[e] += old[e];
  const uint32_t shared = gci::unit_shared(n, UNIT, u, off, VE);
  if (shared == 0) W::store(p, here, 0, W::narrow(v), through);
  else W::store_some(p, shared, VE, W::narrow(v));
}

// Elements of a unit that is at most 16 bytes in either type, so that every store of a wavefront is one run of memory.
template <class In, class OutT>
constexpr int sum_unit() { return In::VE < OutT::VE ? In::VE : OutT::VE; }

template <class In, class OutT, int NV, int P>
__global__ void __launch_bounds__(kThreads) row_sum_kernel(const RowSumArgs<P> a) {
  constexpr int VE = sum_unit<In, OutT>();
  constexpr int AHEAD = 4;   // rows whose loads are in flight together
  typedef AnyUnit<In, VE> U;
  extern __shared__ int2 entries[];   // (id, token) of each group's run and the next one
  const uint64_t block = a.block0 + blockIdx.x;
  if (block >= a.sum_blocks) {
    // rows without a token: a group of lanes takes clear_rows of them
    const uint32_t rows = a.N * a.vocab, lanes = 1u << a.lanes_log2;
    const uint64_t group = (block - a.sum_blocks) * kThreads + threadIdx.x >> a.lanes_log2;
    const uint32_t first = static_cast<uint32_t>(min<uint64_t>(group * a.clear_rows, rows)), last = min(first + a.clear_rows, rows);
    typedef AnyUnit<OutT, VE> W;
    const typename W::T zero = {};
    for (uint32_t r0 = first; r0 < last; r0 += kClearAhead) {
      char* row[kClearAhead];
#pragma unroll
      for (int k = 0; k < kClearAhead; ++k) {
        const uint32_t r = min(r0 + k, last - 1), rank = r / a.vocab, v = r - rank * a.vocab;
        const bool empty = r0 + k < last && !a.present[static_cast<uint64_t>(rank) * a.present_row + v];
        row[k] = empty ? a.dw[rank] + v * (a.H * OutT::ES) : nullptr;
      }
#pragma unroll
      for (int k = 0; k < kClearAhead; ++k) {
        if (!row[k]) continue;
        const uint32_t H = static_cast<uint32_t>(a.H);
        for (uint32_t u = threadIdx.x & (lanes - 1); u < a.units; u += lanes) W::store(row[k], H, W::start(H, u), zero, a.through);
      }
    }
    return;
  }
  const uint64_t q = (block * kThreads + threadIdx.x) >> a.lanes_log2;
  const uint32_t run = static_cast<uint32_t>(a.slices == 1 ? q : q / a.slices);
  const int lanes = 1 << a.lanes_log2, lane = threadIdx.x & (lanes - 1);
  int2* mine = entries + (threadIdx.x >> a.lanes_log2) * (2 * a.run);
  const bool real = run < static_cast<uint32_t>(a.run0[a.N]);
  const int rank = real ? rank_of<P>(a.run0, a.N, static_cast<int32_t>(run)) : 0;
  const int32_t* keys = a.keys + a.at[rank];
  const int64_t n = a.valid[rank];
  const int64_t first = real ? static_cast<int64_t>(run - a.run0[rank]) * a.run : n;
  const auto entries_from = [&](int64_t at, int most) { return static_cast<int>(max<int64_t>(0, min<int64_t>(most, n - at))); };
  int count = entries_from(first, a.run);
  const int staged = entries_from(first, 2 * a.run);
  for (int i = lane; i < staged; i += lanes) mine[i] = int2{keys[first + i], a.perm[a.at[rank] + first + i]};
  const auto key_at = [&](int64_t i) { return i >= 0 && i < n ? keys[i] : -1; };
  // the keys that decide about rows across the run's ends: before it, before the run ahead of it, behind the next run
  const int32_t key_before = key_at(first - 1), key_ahead = key_at(first - a.run - 1), key_behind = key_at(first + 2 * a.run);
  __syncthreads();
  if (count == 0) return;
  int32_t cur = mine[0].x;
  const int32_t last_key = mine[count - 1].x;
  bool began = key_before != cur;      // the current row begins in this run
  bool ended = count == staged || mine[count].x != last_key;   // the last row ends in it
  int i0 = 0;
  if (!began && key_ahead != cur && (last_key != cur || ended)) {
    // the first row began in the run ahead and ends here: that run takes it
    i0 = past(mine, 0, count, cur);
    if (i0 == count) return;
    cur = mine[i0].x;
    began = true;
  }
  if (!ended && (began || last_key != cur) && key_behind != last_key) {
    // the last row begins here and ends in the next run
    count = past(mine, count, staged, last_key);
    ended = true;
  }
  const uint32_t u0 = static_cast<uint32_t>((q - static_cast<uint64_t>(run) * a.slices) * (static_cast<uint64_t>(NV) << a.lanes_log2)) + lane;
  const char* dout = a.dout[rank];
  char* dw = a.dw[rank];
  const uint64_t row_bytes = a.H * In::ES, dw_bytes = a.H * OutT::ES;
  const uint32_t H = static_cast<uint32_t>(a.H);
  uint32_t s[NV];   // first element of each unit; lanes past the row's end read its last one
#pragma unroll
  for (int j = 0; j < NV; ++j) s[j] = U::start(H, u0 + (j << a.lanes_log2));
  float acc[NV][VE] = {};
  const auto flush = [&](bool whole) {
    char* row = dw + cur * dw_bytes;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t u = u0 + (j << a.lanes_log2);
      if (u >= a.units) continue;
      if (began && whole) {
        put_sums<OutT, VE, VE>(row, H, u, 0, acc[j], a.scale, a.accumulate, a.through);
      } else {
        float* p = a.partial + (2 * static_cast<uint64_t>(run) + (began ? 1 : 0)) * a.pitch + static_cast<uint64_t>(u) * VE;
#pragma unroll
        for (int e = 0; e < VE; e += 4) *reinterpret_cast<float4*>(p + e) = float4{acc[j][e], acc[j][e + 1], acc[j][e + 2], acc[j][e + 3]};
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) acc[j][e] = 0.0f;
    }
  };
  // the next rows' loads are in flight while these are added
  const auto fetch = [&](typename U::T (&x)[AHEAD][NV], int i) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const char* row = dout + static_cast<uint32_t>(mine[min(i + k, count - 1)].y) * row_bytes;
#pragma unroll
      for (int j = 0; j < NV; ++j) x[k][j] = U::load(row, H, s[j]);
    }
  };
  const auto take = [&](const typename U::T (&x)[AHEAD][NV], int i) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (i + k >= count) break;
      const int32_t key = mine[i + k].x;
      if (key != cur) {
        flush(true);
        cur = key;
        began = true;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[VE];
        U::widen(x[k][j], v);
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[j][e] += v[e];
      }
    }
  };
  typename U::T xa[AHEAD][NV], xb[AHEAD][NV];
  fetch(xa, i0);
  for (int i = i0; i < count; i += 2 * AHEAD) {
    if (i + AHEAD < count) fetch(xb, i + AHEAD);
    take(xa, i);
    if (i + 2 * AHEAD < count) fetch(xa, i + 2 * AHEAD);
    take(xb, i + AHEAD);
  }
  flush(ended);
  if (began && !ended && u0 == 0) a.long_rows[1 + atomicAdd(&a.long_rows[0], 1)] = static_cast<int32_t>(run);
}

// Adds up the partial sums of the listed rows, 1024 columns per workgroup: four
// groups of 256 lanes take every fourth part (four columns a lane), and their sums
// are added in order.  The list's order does not matter to the results.
constexpr int kJoinThreads = 1024;
constexpr int kJoinGroups = kJoinThreads / 256;

template <class OutT, int VE, int P>
__global__ void __launch_bounds__(kJoinThreads) row_join_kernel(const RowSumArgs<P> a) {
  __shared__ float4 sums[kJoinGroups - 1][256];
  const int group = threadIdx.x / 256, lane = threadIdx.x % 256;
  const uint64_t items = static_cast<uint64_t>(a.long_rows[0]) * a.slices;
  for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint64_t slot = item / a.slices;
    const int32_t run = a.long_rows[1 + slot];
    const int rank = rank_of<P>(a.run0, a.N, run);
    const int32_t* keys = a.keys + a.at[rank];
    const int64_t n = a.valid[rank], end = static_cast<int64_t>(run - a.run0[rank] + 1) * a.run;
    const int32_t key = keys[end - 1];
    int64_t parts = 1;   // and one more for each run behind that starts in the row
    for (int more = kJoinThreads; more == kJoinThreads; parts += more) {
      const int64_t i = end + (parts - 1 + threadIdx.x) * a.run;
      more = __syncthreads_count(i < n && keys[i] == key);
    }
    const uint64_t u = (item - slot * a.slices) * 256 + lane;
    float4 acc{0.0f, 0.0f, 0.0f, 0.0f};
    if (u * 4 < a.units * VE) {
      const float* p = a.partial + 2 * static_cast<uint64_t>(run) * a.pitch + u * 4;
#pragma unroll 8
      for (int64_t i = group; i < parts; i += kJoinGroups) {
        const float4 v = *reinterpret_cast<const float4*>(p + (2 * i + (i == 0 ? 1 : 0)) * a.pitch);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
    }
    if (group > 0) sums[group - 1][lane] = acc;
    __syncthreads();
    if (group == 0 && u * 4 < a.units * VE) {
      float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
      for (int g = 0; g < kJoinGroups - 1; ++g) {
        const float4 t = sums[g][lane];
        v[0] += t.x;
        v[1] += t.y;
        v[2] += t.z;
        v[3] += t.w;
      }
      char* row = a.dw[rank] + static_cast<uint64_t>(key) * a.H * OutT::ES;
      const uint32_t i = static_cast<uint32_t>(u) * 4;   // partial rows: unit after unit
      put_sums<OutT, 4, VE>(row, static_cast<uint32_t>(a.H), i / VE, i % VE, v, a.scale, a.accumulate, a.through);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- host side

template <class In, int NV, int P>
gc_status embedding_impl(const gci::EmbeddingCall& c, EmbeddingArgs<P>& a) {
  const uint64_t per = static_cast<uint64_t>(NV) << a.lanes_log2;
  const uint64_t slices = (a.units + per - 1) / per;
  a.slices = static_cast<uint32_t>(slices);
  if (!fill_blocks<P>(a.tile0, c.tokens, c.nranks, kThreads >> a.lanes_log2, slices)) return GC_ERR_UNSUPPORTED;
  return launch_blocks(embedding_kernel<In, NV, P>, a, a.tile0[c.nranks], kThreads, c.stream);
}

template <class In, int P>
gc_status embedding_typed(const gci::EmbeddingCall& c) {
  EmbeddingArgs<P> a{};
  for (int s = 0; s < c.nranks; ++s) {
    a.w[s] = static_cast<const char*>(c.w[s]);
    a.ids[s] = c.ids[s];
    a.out[s] = static_cast<char*>(c.out[s]);
    a.tok[s] = c.tokens[s];
  }
  a.N = c.nranks;
  a.vocab = static_cast<uint32_t>(c.vocab);
  a.H = c.hidden;
  uint64_t m = c.hidden * In::ES;
  for (int s = 0; s < c.nranks; ++s) m |= c.tokens[s] ? reinterpret_cast<uint64_t>(c.out[s]) : 0;
  a.through = m % kLine == 0;
  a.units = (c.hidden + In::VE - 1) / In::VE;
  a.scale = c.scale;
  while (a.lanes_log2 < 6 && (uint64_t(1) << a.lanes_log2) < a.units) ++a.lanes_log2;
  // units per lane: as many as spread a row evenly over slices of at most four
  const uint64_t waves = (a.units + kWave - 1) / kWave, slices = (waves + 3) / 4, nv = (waves + slices - 1) / slices;
  if (nv <= 1) return embedding_impl<In, 1, P>(c, a);
  if (nv == 2) return embedding_impl<In, 2, P>(c, a);
  return nv == 3 ? embedding_impl<In, 3, P>(c, a) : embedding_impl<In, 4, P>(c, a);
}

template <bool FIRST, bool LAST, int P>
gc_status sort_pass(SortArgs<P>& a, const gci::EmbeddingGeom& g, hipStream_t stream) {
  const size_t bins = size_t(1) << (FIRST ? a.low_bits : a.high_bits);
  void* params[] = {&a};
  const auto go = [&](const void* kernel, size_t lds) {
    return gci::in_launches(g.chunks, kSortThreads, [&](uint32_t first, uint32_t n) {
      a.block0 = first;
      return gci::hip_status(hipLaunchKernel(kernel, dim3(n), dim3(kSortThreads), params, lds, stream));
    });
  };
  const gc_status s = go(reinterpret_cast<const void*>(sort_count_kernel<FIRST, P>), bins * 4);
  return s != GC_OK ? s : go(reinterpret_cast<const void*>(sort_place_kernel<FIRST, LAST, P>), kSortWaves * bins * 4);
}

template <class In, class OutT, int NV, int P>
gc_status row_sums(RowSumArgs<P>& r, bool long_rows, hipStream_t stream) {
  const uint64_t per = static_cast<uint64_t>(NV) << r.lanes_log2, runs = r.run0[r.N];
  r.slices = static_cast<uint32_t>((r.units + per - 1) / per);
  r.sum_blocks = ((runs * r.slices << r.lanes_log2) + kThreads - 1) / kThreads;
  const uint64_t row = r.H * OutT::ES, rows = static_cast<uint64_t>(r.N) * r.vocab;
  // about 64 bytes per lane of a clearing group: 131072 rows of 4096 bf16 of which 4096 tokens use some take 180 us,
  // 224 with 16 or 256 bytes; a million rows of 64 54 us, 62 and 60
  const uint64_t lane_bytes = row >> r.lanes_log2;
  r.clear_rows = static_cast<uint32_t>(std::max<uint64_t>(1, 64 / std::max<uint64_t>(1, lane_bytes)));
  const uint64_t groups = (rows + r.clear_rows - 1) / r.clear_rows;
  const uint64_t clear = r.accumulate ? 0 : ((groups << r.lanes_log2) + kThreads - 1) / kThreads;
  void* params[] = {&r};
  const size_t lds = sizeof(int2) * 2 * r.run * (kThreads >> r.lanes_log2);
  gc_status st = gci::in_launches(r.sum_blocks + clear, kThreads, [&](uint32_t first, uint32_t n) {
    r.block0 = first;
    return gci::hip_status(hipLaunchKernel(reinterpret_cast<const void*>(row_sum_kernel<In, OutT, NV, P>), dim3(n), dim3(kThreads),
                                           params, lds, stream));
  });
  if (st != GC_OK || !long_rows) return st;
  r.slices = static_cast<uint32_t>((r.pitch / 4 + 255) / 256);
  const uint64_t most = std::min<uint64_t>(runs * r.slices, 1024);   // workgroups; two fit a CU
  return gci::hip_status(hipLaunchKernel(reinterpret_cast<const void*>(row_join_kernel<OutT, sum_unit<In, OutT>(), P>), dim3(static_cast<uint32_t>(most)),
                                         dim3(kJoinThreads), params, 0, stream));
}

template <class In, class OutT, int P>
gc_status embedding_backward_typed(const gci::EmbeddingBackwardCall& c) {
  const gci::EmbeddingGeom& g = c.geom;
  char* scratch = static_cast<char*>(c.scratch);
  SortArgs<P> s{};
  RowSumArgs<P> r{};
  int64_t at = 0;
  for (int k = 0; k < c.nranks; ++k) {
    s.ids[k] = c.ids[k];
    s.tok[k] = c.tokens[k];
    s.at[k] = r.at[k] = at;
    r.dout[k] = static_cast<const char*>(c.dout[k]);
    r.dw[k] = static_cast<char*>(c.dw[k]);
    at += c.tokens[k];
    s.tile0[k + 1] = s.tile0[k] + std::max<int32_t>(1, static_cast<int32_t>((c.tokens[k] + g.chunk - 1) / g.chunk));
  }
  for (int k = c.nranks; k < P; ++k) s.tile0[k + 1] = s.tile0[k];
  r.run = g.run;
  fill_blocks<P>(r.run0, c.tokens, c.nranks, r.run);
  bool long_rows = false;   // a row of more tokens than two runs is possible
  for (int k = 0; k < c.nranks; ++k) long_rows |= c.tokens[k] > 2 * r.run;
  s.N = r.N = c.nranks;
  s.chunk = g.chunk;
  s.vocab = r.vocab = static_cast<uint32_t>(c.vocab);
  s.pairs = reinterpret_cast<uint64_t*>(scratch + g.pairs);
  r.keys = s.keys = reinterpret_cast<int32_t*>(scratch + g.keys);
  r.perm = s.perm = reinterpret_cast<int32_t*>(scratch + g.perm);
  s.counts = reinterpret_cast<uint32_t*>(scratch + g.counts);
  r.valid = s.valid = reinterpret_cast<int32_t*>(scratch + g.valid);
  r.present = s.present = reinterpret_cast<uint8_t*>(scratch + g.present);
  r.long_rows = s.long_rows = reinterpret_cast<int32_t*>(scratch + g.long_rows);
  r.partial = reinterpret_cast<float*>(scratch + g.partial);
  r.present_row = s.present_row = static_cast<uint32_t>(g.present_row);
  s.low_bits = g.low_bits;
  s.high_bits = g.bits - g.low_bits;
  gc_status st;
  if (g.chunks == c.nranks) {
    void* params[] = {&s};
    const size_t lds = size_t(kSortWaves) * 4 << std::max(s.low_bits, s.high_bits);
    st = gci::hip_status(hipLaunchKernel(reinterpret_cast<const void*>(sort_alone_kernel<P>), dim3(c.nranks), dim3(kSortThreads), params,
                                         lds, c.stream));
  } else if (s.high_bits == 0) {
    st = sort_pass<true, true, P>(s, g, c.stream);
  } else {
    st = sort_pass<true, false, P>(s, g, c.stream);
    if (st != GC_OK) return st;
    st = sort_pass<false, true, P>(s, g, c.stream);
  }
  if (st != GC_OK) return st;
  r.H = c.hidden;
  constexpr int VE = sum_unit<In, OutT>();
  uint64_t m = c.hidden * OutT::ES;
  for (int k = 0; k < c.nranks; ++k) m |= reinterpret_cast<uint64_t>(c.dw[k]);
  r.through = m % kLine == 0;
  r.units = (c.hidden + VE - 1) / VE;
  r.pitch = gci::embedding_pitch(c.hidden);
  r.scale = c.scale;
  r.accumulate = c.accumulate;
  r.lanes_log2 = 3;
  while (r.lanes_log2 < 8 && (uint64_t(1) << r.lanes_log2) < r.units) ++r.lanes_log2;
  // Two units per lane where that makes no more idle lanes than one: rows of 4096 bf16 245 us against 258, of 8192 480
  // against 490; where it does, one: of 4608 287 us against 326, of 6144 372 against 380 (4 x 8192 rows).
  const uint64_t slices = (r.units + kThreads - 1) / kThreads;
  return slices % 2 ? row_sums<In, OutT, 1, P>(r, long_rows, c.stream) : row_sums<In, OutT, 2, P>(r, long_rows, c.stream);
}

template <class In, class OutT>
gc_status embedding_backward_ranks(const gci::EmbeddingBackwardCall& c) {
  return c.nranks <= 8 ? embedding_backward_typed<In, OutT, 8>(c) : embedding_backward_typed<In, OutT, 64>(c);
}

}  // namespace

namespace gci {

gc_status launch_embedding(const EmbeddingCall& c) {
  if (c.t == GC_BF16) return c.nranks <= 8 ? embedding_typed<InBf16, 8>(c) : embedding_typed<InBf16, 64>(c);
  return c.nranks <= 8 ? embedding_typed<InF32, 8>(c) : embedding_typed<InF32, 64>(c);
}

gc_status launch_embedding_backward(const EmbeddingBackwardCall& c) {
  if (c.t == GC_BF16)
    return c.dw_t == GC_BF16 ? embedding_backward_ranks<InBf16, InBf16>(c) : embedding_backward_ranks<InBf16, InF32>(c);
  return c.dw_t == GC_BF16 ? embedding_backward_ranks<InF32, InBf16>(c) : embedding_backward_ranks<InF32, InF32>(c);
}

}  // namespace gci
