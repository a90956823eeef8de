// The experts' gated feed-forward block and its backward pass for gfx950, on
// the MoE receive layout (blocks of rows by expert).
//
//   forward   gate = x Wg^T, up = x Wu^T, h = silu(gate) up      (one kernel, two accumulators)
//             y = h Wd^T
//   backward  dh = dy Wd; dgate = dh up silu'(gate), dup = dh silu(gate), h again   (one kernel)
//             dx = [dgate dup] [Wg; Wu],  dWd = dy^T h,  [dWg; dWu] = [dgate dup]^T x
//
// Every product is one kernel template over bf16 operands with fp32 MFMA
// accumulators: a workgroup of eight wavefronts owns a tile of TM x 256 outputs
// and walks the summed index in steps of 64 through double-buffered LDS, filled
// by direct global-to-LDS loads.  An operand is stored either with the summed
// index contiguous (rows of 64 values, 128 bytes) or across rows (rows of 256
// values); the second kind is read through the transposing LDS load, so no
// operand is ever laid out again in memory.
//
// The number of rows of each expert is known on the device alone (the routing
// plan's split table): a plan kernel turns it into a table of blocks and row
// tiles, and the grid is sized for the most tiles those rows can make.

#include <algorithm>
#include <type_traits>
#include <utility>

#include "rows.h"

namespace {

using namespace gcdev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef gci::FfnSeg Seg;

constexpr int kGemmThreads = 512;
constexpr int kTileN = 256;
constexpr int kTileK = 64;
constexpr int kXcds = 8;

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 1024;
constexpr int kPlanRanks = 8;     // ranks whose pointers fit one launch's arguments
constexpr int kMaxSegs = 8192;

struct PlanArgs {
  const int64_t* splits;
  int64_t rows[GC_MAX_RANKS];
  const char* x[kPlanRanks];
  const char* dy[kPlanRanks];
  char* saved[kPlanRanks];
  char* y[kPlanRanks];
  const char* w_gate[kPlanRanks];
  const char* w_up[kPlanRanks];
  const char* w_down[kPlanRanks];
  char* dw_gate[kPlanRanks];
  char* dw_up[kPlanRanks];
  char* dw_down[kPlanRanks];
  const char* x_rows;             // decoded x in scratch (null: x[] is read in place)
  Seg* segs;
  int32_t* map;                   // [tiles] block of each row tile, -1 past the last
  int64_t tiles;
  uint64_t x_row, saved_row, y_row;  // bytes
  uint64_t w_bytes, dw_bytes;     // of one expert's gate (= up = down) matrix and its gradient
  int32_t N, E, tile_rows, rank0;
};

// Exclusive prefix over the workgroup of one value per thread.
template <class V>
__device__ __forceinline__ V plan_scan(V v, V* lds) {
  const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
  V x = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const V y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  if (lane == kWave - 1) lds[w] = x;
  __syncthreads();
  V off = 0;
  for (int i = 0; i < w; ++i) off += lds[i];
  __syncthreads();
  return off + x - v;
}

__global__ void __launch_bounds__(kPlanThreads) ffn_plan_kernel(const PlanArgs a) {
  __shared__ int64_t pre[kMaxSegs + 1];  // rows before each expert, over all ranks
  __shared__ int64_t wide[kPlanThreads / kWave];
  __shared__ int32_t narrow[kPlanThreads / kWave];
  __shared__ int64_t base[GC_MAX_RANKS];
  const int nseg = a.N * a.E;
  const int per = (nseg + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(static_cast<int>(threadIdx.x) * per, nseg), hi = min(lo + per, nseg);
  if (threadIdx.x == 0) {
    int64_t run = 0;
    for (int d = 0; d < a.N; ++d) {
      base[d] = run;
      run += a.rows[d];
    }
  }
  int64_t sum = 0;
  for (int i = lo; i < hi; ++i) {
    const int d = i / a.E, e = i - d * a.E;
    int64_t c = 0;  // saturates at the rank's rows, so no sum of entries overflows
    for (int s = 0; s < a.N; ++s) {
      const int64_t v = a.splits[(static_cast<int64_t>(s) * a.N + d) * a.E + e];
      c = min(c + min(max(v, int64_t(0)), a.rows[d]), a.rows[d]);
    }
    pre[i] = c;
    sum += c;
  }
  int64_t run = plan_scan<int64_t>(sum, wide);
  for (int i = lo; i < hi; ++i) {
    const int64_t c = pre[i];
    pre[i] = run;
    run += c;
    if (i == nseg - 1) pre[nseg] = run;
  }
  __syncthreads();
  int32_t tiles = 0;
  for (int i = lo; i < hi; ++i) {
    const int d = i / a.E;
    const int64_t start = min(pre[i] - pre[d * a.E], a.rows[d]), end = min(pre[i + 1] - pre[d * a.E], a.rows[d]);
    tiles += static_cast<int32_t>((end - start + a.tile_rows - 1) / a.tile_rows);
  }
  int32_t tile = plan_scan<int32_t>(tiles, narrow);
  for (int i = lo; i < hi; ++i) {
    const int d = i / a.E, e = i - d * a.E, q = d - a.rank0;
    const int64_t start = min(pre[i] - pre[d * a.E], a.rows[d]), end = min(pre[i + 1] - pre[d * a.E], a.rows[d]);
    const int32_t n = static_cast<int32_t>((end - start + a.tile_rows - 1) / a.tile_rows);
    if (q >= 0 && q < kPlanRanks) {
      Seg s;
      s.row = base[d] + start;
      s.x = a.x_rows ? a.x_rows + s.row * a.x_row : a.x[q] + start * a.x_row;
      s.dy = a.dy[q] + start * a.y_row;
      s.saved = a.saved[q] + start * a.saved_row;
      s.y = a.y[q] + start * a.y_row;
      s.w_gate = a.w_gate[q] + e * a.w_bytes;
      s.w_up = a.w_up[q] + e * a.w_bytes;
      s.w_down = a.w_down[q] + e * a.w_bytes;
      s.dw_gate = a.dw_gate[q] + e * a.dw_bytes;
      s.dw_up = a.dw_up[q] + e * a.dw_bytes;
      s.dw_down = a.dw_down[q] + e * a.dw_bytes;
      s.rows = static_cast<int32_t>(end - start);
      s.tile0 = tile;
      a.segs[i] = s;
      for (int32_t t = 0; t < n; ++t) a.map[tile + t] = i;
    }
    tile += n;
    if (i == nseg - 1) narrow[0] = tile;
  }
  __syncthreads();
  for (int64_t t = narrow[0] + threadIdx.x; t < a.tiles; t += kPlanThreads) a.map[t] = -1;
}

// ------------------------------------------------------------------ products

enum Product { kGateUp, kDown, kDh, kDx, kDwDown, kDwGateUp };

struct GemmArgs {
  const Seg* segs;
  const int32_t* map;
  char* h;                 // scratch [rows][F] bf16
  char* g;                 // scratch [rows][2F] bf16: dgate then dup
  uint32_t mtiles;         // row tiles (row products) or output row tiles of one expert (weight gradients)
  uint32_t ntiles;
  uint64_t H, F;
  uint64_t saved_row;
  uint32_t segs_n;
};

// Where one operand's tile comes from.  kc: the summed index is contiguous in
// memory (rows x K); else each row holds one summed index.
struct Side {
  const char* p;
  const char* p2;          // second half: of the tile's rows (kc) or of the summed index
  uint64_t ld;             // bytes per stored row
  int32_t rows;            // valid rows of the tile (kc), or valid values of a row (else)
};

// The plan's tables were written by an earlier kernel and do not change here:
// read through the constant address space they come by scalar loads and stay
// in scalar registers, where the operands' buffer descriptors need them (the
// compiler cannot tell by itself, because the kernel also writes memory).
typedef const __attribute__((address_space(4))) Seg ConstSeg;
__device__ __forceinline__ ConstSeg* as_constant(const Seg* p) { return (ConstSeg*)(uintptr_t)p; }
__device__ __forceinline__ const __attribute__((address_space(4))) int32_t* as_constant(const int32_t* p) {
  return (const __attribute__((address_space(4))) int32_t*)(uintptr_t)p;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// One tile of a product: its operands, the summed length, where it goes.
struct Tile {
  ConstSeg* sg;
  Side A, B;
  uint32_t K;              // below 2^31
  int64_t m0, n0;
};

constexpr uint32_t kOutside = 0x80000000u;  // past every descriptor's range: the load gives zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const char* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, 0x7FFFFFFF, 0x00020000);
}

__device__ __forceinline__ void lds_load(const char* base, char* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(base), (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
}

// Tile of ROWS rows x 64 summed values: 16-byte chunk c of row r sits at chunk
// c ^ ((r >> 1) & 7) of the row's 128 bytes, so that 16 lanes reading one
// chunk of 16 rows touch all 64 banks.  A wavefront's load covers eight rows.
template <int ROWS, bool HALVES>
__device__ __forceinline__ void load_kc(char* dst, const Side& s, uint32_t k0, uint32_t K, int w, int lane) {
  constexpr int L = ROWS / 64;  // loads per wavefront
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int q = w * L + i, r = q * 8 + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    const bool second = HALVES && q * 8 >= ROWS / 2;
    const int rr = second ? r - ROWS / 2 : r;
    const bool ok = rr < s.rows && k0 + c * 8 < K;
    const uint32_t off = static_cast<uint32_t>(rr * s.ld) + c * 16;
    lds_load((second ? s.p2 : s.p) + static_cast<uint64_t>(k0) * 2, dst + q * 1024, ok ? off : kOutside);
  }
}

// Tile of 64 summed indices x 256 values: 512-byte rows whose 32-byte unit u
// sits at u ^ 2 (k & 3), so that the four rows a transposing read takes
// together lie in different banks.  A wavefront's load covers two rows.
__device__ __forceinline__ void load_ks(char* dst, const Side& s, uint32_t k0, uint32_t K, uint32_t K1, int w, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = w * 4 + i, kr = q * 2 + (lane >> 5);
    const int c = (lane & 31) ^ (4 * (kr & 3));
    const uint32_t k = k0 + q * 2;  // even, as is K1: a pair of rows lies in one half
    const char* base = k < K1 ? s.p + k * s.ld : s.p2 + (k - K1) * s.ld;
    const bool ok = k0 + kr < K && c * 8 < s.rows;
    const uint32_t off = static_cast<uint32_t>((lane >> 5) * s.ld) + c * 16;
    lds_load(base, dst + q * 1024, ok ? off : kOutside);
  }
}

// A lane's eight summed values (16 kk + 8 (lane / 32) ..) of row r0 + lane % 32.
__device__ __forceinline__ bf16x8 frag_kc(const char* t, int r0, int kk, int lane) {
  const int r = r0 + (lane & 31);
  return *reinterpret_cast<const bf16x8*>(t + r * 128 + (((kk * 2 + (lane >> 5)) ^ ((r >> 1) & 7)) * 16));
}

// The same from a tile stored across rows, block of 32 values at 32 b: each
// group of 16 lanes reads 4 rows x 16 values and receives them transposed.
__device__ __forceinline__ bf16x8 frag_ks(const char* t, int b, int kk, int lane) {
  typedef __attribute__((address_space(3))) bf16x4 L;
  const int i = lane & 15, q = lane >> 4;
  const int k = kk * 16 + (q >> 1) * 8 + (i >> 2);
  const int u = (2 * b + (q & 1)) ^ (2 * (i >> 2));
  const char* p = t + k * 512 + u * 32 + (i & 3) * 8;
  const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((L*)p);
  const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((L*)(p + 4 * 512));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A 32 x 32 block of results: lane l holds output row l % 32 and, of its 32
// columns, 8 j + 4 (l / 32) + i as v[4 j + i].  For wide stores the two halves
// of the wavefront trade: afterwards lane l holds columns 8 (2 p + l / 32) ..
// + 7, one 16-byte vector of bf16 for p = 0 and one for p = 1.
__device__ __forceinline__ void swap_halves(uint32_t& x, uint32_t& y) {
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  x = r[0];
  y = r[1];
}

__device__ __forceinline__ void pack_block(const f32x16& v, u32x4 (&o)[2]) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t a0 = bf16_bits(v[8 * p]) | (bf16_bits(v[8 * p + 1]) << 16);
    uint32_t a1 = bf16_bits(v[8 * p + 2]) | (bf16_bits(v[8 * p + 3]) << 16);
    uint32_t b0 = bf16_bits(v[8 * p + 4]) | (bf16_bits(v[8 * p + 5]) << 16);
    uint32_t b1 = bf16_bits(v[8 * p + 6]) | (bf16_bits(v[8 * p + 7]) << 16);
    swap_halves(a0, b0);
    swap_halves(a1, b1);
    o[p] = u32x4{a0, a1, b0, b1};
  }
}

__device__ __forceinline__ void unpack_block(const u32x4 (&o)[2], float (&v)[16]) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t w[4] = {o[p][0], o[p][1], o[p][2], o[p][3]};
    swap_halves(w[0], w[2]);
    swap_halves(w[1], w[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * p + 2 * i] = __uint_as_float(w[i] << 16);
      v[8 * p + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// bf16 store of a block: columns n0 .. n0 + 31 of the lane's row (ok: the row exists).
__device__ __forceinline__ void store_block(char* row, uint64_t n0, uint64_t N, bool ok, int lane, const f32x16& v) {
  u32x4 o[2];
  pack_block(v, o);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint64_t n = n0 + 8 * (2 * p + (lane >> 5));
    if (ok && n < N) *reinterpret_cast<u32x4*>(row + n * 2) = o[p];
  }
}

// 8-bit store of a block, which is one scale block of the row: values at
// column c0 of the row's n, all 32 of them inside (32 divides n and c0).
__device__ __forceinline__ void store_block8(char* row, uint64_t n, uint64_t c0, bool ok, int lane, const f32x16& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, mx8_magnitude(v[i]));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
  const int e = mx8_exponent(m);
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    c[j] = mx8_codes(mx8_scaled(v[4 * j], e), mx8_scaled(v[4 * j + 1], e), mx8_scaled(v[4 * j + 2], e),
                     mx8_scaled(v[4 * j + 3], e));
  swap_halves(c[0], c[1]);
  swap_halves(c[2], c[3]);
  if (!ok) return;
#pragma unroll
  for (int p = 0; p < 2; ++p)
    *reinterpret_cast<u32x2*>(row + c0 + 8 * (2 * p + (lane >> 5))) = u32x2{c[2 * p], c[2 * p + 1]};
  if (lane < 32) row[n + c0 / 32] = static_cast<char>(e + 127);
}

__device__ __forceinline__ void load_block8(const char* row, uint64_t n, uint64_t c0, int lane, float (&v)[16]) {
  const float s = mx8_scale(*reinterpret_cast<const uint8_t*>(row + n + c0 / 32));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[4];
    mx8_values(*reinterpret_cast<const uint32_t*>(row + c0 + 8 * j + 4 * (lane >> 5)), s, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * j + i] = f[i];
  }
}

__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// Instruction classes of the scheduling barriers.
constexpr int kMfma = 0x8, kDsRead = 0x100;

// One matrix instruction, then N LDS reads.
template <int N>
__device__ __forceinline__ void group_pair() {
  __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
  if constexpr (N > 0) __builtin_amdgcn_sched_group_barrier(kDsRead, N, 0);
}

// READS reads spread evenly behind the MM matrix instructions.
template <int READS, int MM, int... M>
__device__ __forceinline__ void group_pairs(std::integer_sequence<int, M...>) {
  (group_pair<(READS * (M + 1)) / MM - (READS * M) / MM>(), ...);
}

enum SavedKind { kNoSaved, kSaved16, kSaved8 };

// One tile of one product.  MB: 32-row blocks per wavefront (two wavefronts
// along the rows, four along the 256 columns, two blocks of columns each).
// SAVED: the checkpoint's type (kGateUp, kDh).  F32OUT: fp32 weight gradients.
template <int KIND, int MB, int SAVED, bool F32OUT>
__global__ void __launch_bounds__(kGemmThreads, MB == 1 ? 4 : 2) ffn_gemm_kernel(const GemmArgs a) {
  constexpr int TM = 64 * MB;
  constexpr bool WGRAD = KIND == kDwDown || KIND == kDwGateUp;
  constexpr bool A_KC = !WGRAD;
  constexpr bool B_KC = KIND == kGateUp || KIND == kDown;
  static_assert(!WGRAD || MB == 4, "tiles across rows are 256 wide");
  __shared__ __align__(1024) char A0[TM * 128];
  __shared__ __align__(1024) char A1[TM * 128];
  __shared__ __align__(1024) char B0[kTileN * 128];
  __shared__ __align__(1024) char B1[kTileN * 128];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 2, wn = w & 3;
  const uint64_t H = a.H, F = a.F;

  const uint32_t total = a.mtiles * a.ntiles * (WGRAD ? a.segs_n : 1u);  // below 2^31, checked on the host

  // Tile t of the product.  Tiles are numbered four row tiles deep, so that
  // the ones that run together on an XCD share operands in its L2.  False for a
  // row tile past the blocks' last.
  auto find = [&](uint32_t t, Tile& r) -> bool {
    constexpr uint32_t GM = 4;
    const uint32_t per = a.mtiles * a.ntiles;
    const uint32_t s = WGRAD ? uniform(t / per) : 0;
    const uint32_t tt = t - s * per;
    const uint32_t grp = uniform(tt / (GM * a.ntiles)), in = tt - grp * GM * a.ntiles;
    const uint32_t depth = std::min(GM, a.mtiles - grp * GM);
    const uint32_t nt = depth == GM ? in / GM : uniform(in / depth), mt = grp * GM + in - nt * depth;
    const int32_t seg = WGRAD ? static_cast<int32_t>(s) : as_constant(a.map)[mt];
    if (seg < 0) return false;
    const ConstSeg& sg = as_constant(a.segs)[seg];
    r.sg = &sg;
    const int64_t m0 = r.m0 = static_cast<int64_t>(WGRAD ? mt : mt - sg.tile0) * TM;
    const int64_t n0 = r.n0 = static_cast<int64_t>(nt) * (KIND == kGateUp ? kTileN / 2 : kTileN);
    Side &A = r.A, &B = r.B;
    const auto left = [](int64_t most, uint64_t n) { return static_cast<int32_t>(std::min<int64_t>(most, n)); };
    if constexpr (KIND == kGateUp) {
      r.K = H;
      A = {sg.x + m0 * H * 2, nullptr, H * 2, left(TM, sg.rows - m0)};
      B = {sg.w_gate + n0 * H * 2, sg.w_up + n0 * H * 2, H * 2, left(kTileN / 2, F - n0)};
    } else if constexpr (KIND == kDown) {
      r.K = F;
      A = {a.h + (sg.row + m0) * F * 2, nullptr, F * 2, left(TM, sg.rows - m0)};
      B = {sg.w_down + n0 * F * 2, nullptr, F * 2, left(kTileN, H - n0)};
    } else if constexpr (KIND == kDh) {
      r.K = H;
      A = {sg.dy + m0 * H * 2, nullptr, H * 2, left(TM, sg.rows - m0)};
      B = {sg.w_down + n0 * 2, nullptr, F * 2, left(kTileN, F - n0)};
    } else if constexpr (KIND == kDx) {
      r.K = 2 * F;
      A = {a.g + (sg.row + m0) * F * 4, nullptr, F * 4, left(TM, sg.rows - m0)};
      B = {sg.w_gate + n0 * 2, sg.w_up + n0 * 2, H * 2, left(kTileN, H - n0)};
    } else if constexpr (KIND == kDwDown) {
      r.K = sg.rows;
      A = {sg.dy + m0 * 2, nullptr, H * 2, left(TM, H - m0)};
      B = {a.h + (sg.row * F + n0) * 2, nullptr, F * 2, left(kTileN, F - n0)};
    } else {
      r.K = sg.rows;
      A = {a.g + (sg.row * 2 * F + m0) * 2, nullptr, F * 4, left(TM, 2 * F - m0)};
      B = {sg.x + n0 * 2, nullptr, H * 2, left(kTileN, H - n0)};
    }
    return true;
  };
  // The workgroup's tiles: every gridDim.x-th, the ones of one round next to
  // each other on each XCD (blocks go round the XCDs).
  uint32_t next = blockIdx.x % kXcds * (gridDim.x / kXcds) + blockIdx.x / kXcds;
  auto advance = [&](Tile& r) -> bool {
    for (; next < total; next += gridDim.x)
      if (find(next, r)) {
        next += gridDim.x;
        return true;
      }
    return false;
  };

  f32x16 acc[MB][2];
  auto load = [&](char* da, char* db, const Tile& r, uint32_t k0) {
    if constexpr (A_KC) load_kc<TM, false>(da, r.A, k0, r.K, w, lane);
    else load_ks(da, r.A, k0, r.K, ~0u, w, lane);
    if constexpr (B_KC) load_kc<kTileN, KIND == kGateUp>(db, r.B, k0, r.K, w, lane);
    else load_ks(db, r.B, k0, r.K, KIND == kDx ? static_cast<uint32_t>(F) : ~0u, w, lane);
  };
  // One step of 64 summed values: the fragments of each 16 are read while the
  // matrix cores work on the 16 before.  The group barriers pin that order; left
  // alone, the compiler reads each fragment just before its use, to save
  // registers, and every read's latency shows.
  auto compute = [&](const char* ta, const char* tb) {
    constexpr int STEPS = kTileK / 16, MM = 2 * MB;
    constexpr int READS = MB * (A_KC ? 1 : 2) + 2 * (B_KC ? 1 : 2);
    bf16x8 fa[2][MB], fb[2][2];
    auto fragments = [&](int s, int kk) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = KIND == kGateUp ? wn + 4 * j : wn * 2 + j;  // 32-column block
        if constexpr (B_KC) fb[s][j] = frag_kc(tb, b * 32, kk, lane);
        else fb[s][j] = frag_ks(tb, b, kk, lane);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if constexpr (A_KC) fa[s][i] = frag_kc(ta, (wm * MB + i) * 32, kk, lane);
        else fa[s][i] = frag_ks(ta, wm * MB + i, kk, lane);
      }
    };
    fragments(0, 0);
    __builtin_amdgcn_sched_group_barrier(kDsRead, READS, 0);
#pragma unroll
    for (int kk = 0; kk < STEPS; ++kk) {
      if (kk + 1 < STEPS) fragments((kk + 1) & 1, kk + 1);
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[kk & 1][j], fa[kk & 1][i], acc[i][j], 0, 0, 0);
      if (kk + 1 < STEPS) {
        group_pairs<READS, MM>(std::make_integer_sequence<int, MM>{});
      } else {
        __builtin_amdgcn_sched_group_barrier(kMfma, MM, 0);
      }
    }
  };

  Tile cur;
  bool more = advance(cur);
  if (!more) return;
  load(A0, B0, cur, 0);
  __syncthreads();
  while (more) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
    Tile then;
    more = advance(then);
    // Two steps a turn, so that each buffer is known at compile time (the
    // compiler then lets reads of one pass loads into the other).  The last
    // turn already loads the next tile's first step, which the epilogue hides.
    const uint32_t K = cur.K;
    uint32_t k0 = 0;
    do {
      if (k0 + kTileK < K) load(A1, B1, cur, k0 + kTileK);
      compute(A0, B0);
      __syncthreads();
      const bool last = k0 + 2 * kTileK >= K;
      if (!last) load(A0, B0, cur, k0 + 2 * kTileK);
      else if (more) load(A0, B0, then, 0);
      if (k0 + kTileK < K) compute(A1, B1);
      __syncthreads();
      k0 += 2 * kTileK;
    } while (k0 < K);
    ConstSeg& sg = *cur.sg;
    const int64_t m0 = cur.m0, n0 = cur.n0;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int64_t m = m0 + (wm * MB + i) * 32 + (lane & 31);
      if constexpr (KIND == kGateUp) {
        const bool row = m < sg.rows;
        const uint64_t n = n0 + wn * 32;
        f32x16 hv;
#pragma unroll
        for (int e = 0; e < 16; ++e) hv[e] = acc[i][0][e] * sigmoid(acc[i][0][e]) * acc[i][1][e];
        store_block(a.h + (sg.row + m) * F * 2, n, F, row, lane, hv);
        if constexpr (SAVED == kSaved16) {
          store_block(sg.saved + m * a.saved_row, n, F, row, lane, acc[i][0]);
          store_block(sg.saved + m * a.saved_row + F * 2, n, F, row, lane, acc[i][1]);
        } else if constexpr (SAVED == kSaved8) {
          char* const out = sg.saved + m * a.saved_row;
          store_block8(out, 2 * F, n, row && n < F, lane, acc[i][0]);
          store_block8(out, 2 * F, F + n, row && n < F, lane, acc[i][1]);
          if (row && n == 0 && lane < 32)  // zeros behind the scales
            for (uint64_t p = 2 * F + 2 * F / 32; p < a.saved_row; ++p) out[p] = 0;
        }
      } else if constexpr (KIND == kDh) {
        const bool row = m < sg.rows;
        const char* in = sg.saved + static_cast<uint64_t>(std::min<int64_t>(m, sg.rows - 1)) * a.saved_row;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint64_t n = n0 + wn * 64 + j * 32;
          if (n >= F) continue;
          float gate[16], up[16];
          if constexpr (SAVED == kSaved16) {
            u32x4 gv[2], uv[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint64_t c = std::min<uint64_t>(n + 8 * (2 * p + (lane >> 5)), F - 8);
              gv[p] = *reinterpret_cast<const u32x4*>(in + c * 2);
              uv[p] = *reinterpret_cast<const u32x4*>(in + (F + c) * 2);
            }
            unpack_block(gv, gate);
            unpack_block(uv, up);
          } else {
            load_block8(in, 2 * F, n, lane, gate);
            load_block8(in, 2 * F, F + n, lane, up);
          }
          f32x16 hv, dg, du;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float g = gate[e], u = up[e], d = acc[i][j][e];
            const float s = sigmoid(g), act = g * s;
            hv[e] = act * u;
            dg[e] = d * u * (s * (1.0f + g * (1.0f - s)));
            du[e] = d * act;
          }
          store_block(a.h + (sg.row + m) * F * 2, n, F, row, lane, hv);
          store_block(a.g + (sg.row + m) * F * 4, n, F, row, lane, dg);
          store_block(a.g + (sg.row + m) * F * 4 + F * 2, n, F, row, lane, du);
        }
      } else if constexpr (!WGRAD) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          store_block(sg.y + m * H * 2, n0 + wn * 64 + j * 32, H, m < sg.rows, lane, acc[i][j]);
      } else {
        constexpr int ES = F32OUT ? 4 : 2;
        const uint64_t M = KIND == kDwDown ? H : 2 * F, N = KIND == kDwDown ? F : H;
        const bool row = static_cast<uint64_t>(m) < M;
        char* out;
        if constexpr (KIND == kDwDown) out = sg.dw_down + m * N * ES;
        else out = static_cast<uint64_t>(m) < F ? sg.dw_gate + m * N * ES : sg.dw_up + (m - static_cast<int64_t>(F)) * N * ES;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint64_t n = n0 + wn * 64 + j * 32;
          if constexpr (F32OUT) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint64_t c = n + 8 * q + 4 * (lane >> 5);
              if (row && c < N)
                *reinterpret_cast<u32x4*>(out + c * 4) =
                    u32x4{__float_as_uint(acc[i][j][4 * q]), __float_as_uint(acc[i][j][4 * q + 1]),
                          __float_as_uint(acc[i][j][4 * q + 2]), __float_as_uint(acc[i][j][4 * q + 3])};
            }
          } else {
            store_block(out, n, N, row, lane, acc[i][j]);
          }
        }
      }
    }
    cur = then;
  }
}

// ------------------------------------------------------------------ host side

uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

template <class Kern, class A>
gc_status launch(Kern kernel, const A& args, uint64_t grid, uint32_t threads, hipStream_t stream) {
  void* params[] = {const_cast<A*>(&args)};
  return gci::hip_status(hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(static_cast<uint32_t>(grid)),
                                         dim3(threads), params, 0, stream));
}

// Workgroups of a product: as many as run at once (`per_cu` on each of the 256
// CUs), or one per tile where there are fewer, a whole number per XCD.
uint64_t grid_for(int64_t tiles, int per_cu) {
  return static_cast<uint64_t>(std::min<int64_t>((tiles + kXcds - 1) / kXcds * kXcds, 256 * per_cu));
}

int64_t ceil_div(uint64_t a, uint64_t b) { return static_cast<int64_t>((a + b - 1) / b); }

gc_status plan(const gci::FfnCall& c, const gci::FfnGeom& g) {
  char* const base = static_cast<char*>(c.scratch);
  for (int r0 = 0; r0 < c.nranks; r0 += kPlanRanks) {
    PlanArgs a{};
    a.splits = c.splits;
    for (int d = 0; d < c.nranks; ++d) a.rows[d] = c.rows[d];
    for (int q = 0; q < kPlanRanks && r0 + q < c.nranks; ++q) {
      const int d = r0 + q;
      a.x[q] = static_cast<const char*>(c.x[d]);
      a.dy[q] = c.dy ? static_cast<const char*>(c.dy[d]) : nullptr;
      a.saved[q] = c.saved ? static_cast<char*>(c.saved[d]) : nullptr;
      a.y[q] = static_cast<char*>(c.y[d]);
      a.w_gate[q] = static_cast<const char*>(c.w_gate[d]);
      a.w_up[q] = static_cast<const char*>(c.w_up[d]);
      a.w_down[q] = static_cast<const char*>(c.w_down[d]);
      if (c.dw_gate) {
        a.dw_gate[q] = static_cast<char*>(c.dw_gate[d]);
        a.dw_up[q] = static_cast<char*>(c.dw_up[d]);
        a.dw_down[q] = static_cast<char*>(c.dw_down[d]);
      }
    }
    a.x_rows = c.x_t == GC_MX8 ? base + g.x : nullptr;
    a.segs = reinterpret_cast<Seg*>(base);
    a.map = reinterpret_cast<int32_t*>(base + g.map);
    a.tiles = g.tiles;
    a.x_row = c.hidden * 2;
    a.saved_row = c.saved_t == GC_MX8 ? gci::mx8_row_bytes(2 * c.inter) : c.inter * 4;
    a.y_row = c.hidden * 2;
    a.w_bytes = c.hidden * c.inter * 2;
    a.dw_bytes = c.hidden * c.inter * (c.dw_t == GC_FP32 ? 4 : 2);
    a.N = c.nranks;
    a.E = c.experts_per_rank;
    a.tile_rows = g.tile_rows;
    a.rank0 = r0;
    const gc_status st = launch(ffn_plan_kernel, a, 1, kPlanThreads, c.stream);
    if (st != GC_OK) return st;
  }
  return GC_OK;
}

// 8-bit x rows, decoded into scratch for the products.
gc_status decode_x(const gci::FfnCall& c, const gci::FfnGeom& g) {
  if (c.x_t != GC_MX8) return GC_OK;
  void* dst[GC_MAX_RANKS];
  char* p = static_cast<char*>(c.scratch) + g.x;
  for (int d = 0; d < c.nranks; ++d) {
    dst[d] = p;
    p += c.rows[d] * c.hidden * 2;
  }
  gci::Mx8Call u{c.x, dst, c.rows, c.nranks, c.hidden, GC_BF16, true, c.stream};
  return gci::launch_mx8(u);
}

GemmArgs gemm_args(const gci::FfnCall& c, const gci::FfnGeom& g) {
  char* const base = static_cast<char*>(c.scratch);
  GemmArgs a{};
  a.segs = reinterpret_cast<const Seg*>(base);
  a.map = reinterpret_cast<const int32_t*>(base + g.map);
  a.h = base + g.h;
  a.g = base + g.g;
  a.H = c.hidden;
  a.F = c.inter;
  a.saved_row = c.saved_t == GC_MX8 ? gci::mx8_row_bytes(2 * c.inter) : c.inter * 4;
  a.segs_n = g.segs;
  return a;
}

template <int KIND, int SAVED>
gc_status row_product(GemmArgs a, const gci::FfnGeom& g, int64_t ntiles, hipStream_t stream) {
  a.mtiles = g.tiles;
  a.ntiles = ntiles;
  const uint64_t grid = grid_for(a.mtiles * a.ntiles, g.tile_rows == 64 ? 2 : 1);
  if (g.tile_rows == 256) return launch(ffn_gemm_kernel<KIND, 4, SAVED, false>, a, grid, kGemmThreads, stream);
  if (g.tile_rows == 128) return launch(ffn_gemm_kernel<KIND, 2, SAVED, false>, a, grid, kGemmThreads, stream);
  return launch(ffn_gemm_kernel<KIND, 1, SAVED, false>, a, grid, kGemmThreads, stream);
}

template <int KIND>
gc_status weight_product(GemmArgs a, uint64_t M, uint64_t N, bool f32, hipStream_t stream) {
  a.mtiles = ceil_div(M, 256);
  a.ntiles = ceil_div(N, kTileN);
  const uint64_t grid = grid_for(a.mtiles * a.ntiles * a.segs_n, 1);
  if (f32) return launch(ffn_gemm_kernel<KIND, 4, kNoSaved, true>, a, grid, kGemmThreads, stream);
  return launch(ffn_gemm_kernel<KIND, 4, kNoSaved, false>, a, grid, kGemmThreads, stream);
}

}  // namespace

namespace gci {

gc_status launch_moe_ffn(const FfnCall& c) {
  const FfnGeom g = ffn_geom(c.rows, c.nranks, c.experts_per_rank, c.hidden, c.inter, c.x_t, false);
  if (g.rows == 0) return GC_OK;
  gc_status st = plan(c, g);
  if (st == GC_OK) st = decode_x(c, g);
  if (st != GC_OK) return st;
  const GemmArgs a = gemm_args(c, g);
  const int64_t nt = ceil_div(c.inter, kTileN / 2);
  if (!c.saved) st = row_product<kGateUp, kNoSaved>(a, g, nt, c.stream);
  else if (c.saved_t == GC_MX8) st = row_product<kGateUp, kSaved8>(a, g, nt, c.stream);
  else st = row_product<kGateUp, kSaved16>(a, g, nt, c.stream);
  if (st != GC_OK) return st;
  return row_product<kDown, kNoSaved>(a, g, ceil_div(c.hidden, kTileN), c.stream);
}

gc_status launch_moe_ffn_backward(const FfnCall& c) {
  const FfnGeom g = ffn_geom(c.rows, c.nranks, c.experts_per_rank, c.hidden, c.inter, c.x_t, true);
  gc_status st = plan(c, g);
  if (st == GC_OK) st = decode_x(c, g);
  if (st != GC_OK) return st;
  const GemmArgs a = gemm_args(c, g);
  if (g.rows > 0) {
    const int64_t nt = ceil_div(c.inter, kTileN);
    st = c.saved_t == GC_MX8 ? row_product<kDh, kSaved8>(a, g, nt, c.stream) : row_product<kDh, kSaved16>(a, g, nt, c.stream);
    if (st == GC_OK) st = row_product<kDx, kNoSaved>(a, g, ceil_div(c.hidden, kTileN), c.stream);
    if (st != GC_OK) return st;
  }
  st = weight_product<kDwDown>(a, c.hidden, c.inter, c.dw_t == GC_FP32, c.stream);
  if (st != GC_OK) return st;
  return weight_product<kDwGateUp>(a, 2 * c.inter, c.hidden, c.dw_t == GC_FP32, c.stream);
}

}  // namespace gci
