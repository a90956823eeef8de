// The experts' gated feed-forward block and its backward pass for gfx950, on
// the MoE receive layout (blocks of rows by expert).
//
//   forward   gate = x Wg^T, up = x Wu^T, h = silu(gate) up      (one kernel, two accumulators)
//             y = h Wd^T
//   backward  dh = dy Wd; dgate = dh up silu'(gate), dup = dh silu(gate), h again   (one kernel)
//             dx = [dgate dup] [Wg; Wu],  dWd = dy^T h,  [dWg; dWu] = [dgate dup]^T x
//
// Every product is one kernel template over bf16 operands with fp32 MFMA
// accumulators: a workgroup owns tiles of TM x 256 outputs
// and walks the summed index in steps of 64 through double-buffered LDS, filled
// by direct global-to-LDS loads.  An operand is stored either with the summed
// index contiguous (rows of 64 values, 128 bytes) or across rows (rows of 256
// values); the second kind is read through the transposing LDS load, so no
// operand is ever laid out again in memory.
//
// h, dgate and dup are kept as bf16 between the products: one more rounding of half
// a step, of the same size as the result's own, averaged over the rows and sums
// that a value enters.  With few rows per expert little is averaged, and the
// products wait for the weights anyway: there (SPLIT) each is kept as the sum of two
// bf16 values, the second the first's rounding error (within 2^-17 of the value
// together).  A row product's tile then holds 32 rows and 32 rests, whose results
// its two halves add; a weight gradient sums over the rests and then the rows.
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
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef gci::FfnSeg Seg;

constexpr int kTileN = 256;
constexpr int kWaves = 8;
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
    for (int s0 = 0; s0 < a.N; s0 += 8) {  // eight loads in flight
      int64_t v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = a.splits[(static_cast<int64_t>(min(s0 + q, a.N - 1)) * a.N + d) * a.E + e];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (s0 + q < a.N) c = min(c + min(max(v[q], int64_t(0)), a.rows[d]), a.rows[d]);
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

// Where one operand's tile comes from.  kc: the summed index is contiguous in
// memory (rows x K); else each stored row holds one summed index.
struct Side {
  const char* p;
  const char* p2;          // second half: of the tile's rows (kc) or of the summed index
  int32_t n;               // valid rows of the tile (kc), or valid values of a stored row (else)
};

// One tile of a product: its operands, the summed length, where it goes.
struct Tile {
  ConstSeg* sg;
  Side A, B;
  uint32_t K;              // below 2^31
  uint32_t part, sum;      // split operands: the length of each part (a multiple of 64), the summed values in it
  int64_t m0, n0;
};

// x's operands if c, else y's; field by field, so that they stay in registers.
__device__ __forceinline__ Side pick(bool c, const Side& x, const Side& y) {
  return {c ? x.p : y.p, c ? x.p2 : y.p2, c ? x.n : y.n};
}

// One step's loads: summed indices from k0 of K.
struct Load {
  Side a, b;
  uint32_t k0, K, part, sum;
};

constexpr uint32_t kOutside = 0x80000000u;  // past every descriptor's range, whatever is added: the load gives zeros

// Loads of one operand's tile by eight wavefronts, straight from memory into LDS
// (1 KiB per wavefront and instruction, 16 bytes per lane).  Rows, columns and
// summed indices outside the operand come as zeros: the buffer descriptor ends
// behind the last valid row, and a lane outside its row gets an offset past it.
//
// kc: ROWS rows x 64 summed values; chunk c (16 bytes) of row r sits at chunk
// c ^ ((r >> 1) & 7) of the row's 128 bytes, so that 16 lanes reading one chunk
// of 16 rows touch all 64 banks.  An instruction covers eight rows.
// else: 64 summed indices x 256 values; the 32-byte unit u of row k sits at
// u ^ 2 (k & 3), so that the four rows a transposing read takes together lie in
// different banks.  An instruction covers two rows.
//
// Either way an instruction's lanes differ between tiles only by a multiple of
// the rows skipped and by the parity of its number, so two lane offsets serve all.
template <bool KC, int ROWS, bool HALVES>
struct Loader {
  static constexpr int L = KC ? ROWS / 8 / kWaves : 32 / kWaves;  // instructions per wavefront
  uint32_t ld;      // bytes per stored row
  uint32_t off[2];  // lane offset by parity
  uint32_t c8[2];   // the lane's first value in its stored row's part
  int q0;           // first instruction

  __device__ __forceinline__ Loader(uint64_t stored, int w, int lane) : ld(static_cast<uint32_t>(stored)), q0(w * L) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int q = q0 + e, r = KC ? lane >> 3 : lane >> 5;
      const int c = KC ? (lane & 7) ^ (((q * 8 + r) >> 1) & 7) : (lane & 31) ^ (4 * ((q * 2 + r) & 3));
      off[e] = r * ld + c * 16;
      c8[e] = c * 8;
    }
  }

  // The step's summed indices start at k0 of K; for !KC those from K1 on come from p2.
  // Instructions [I0, I1) of it.
  template <int I0 = 0, int I1 = L>
  __device__ __forceinline__ void run(char* dst, const Side& s, uint32_t k0, uint32_t K, uint32_t K1) const {
    const uint32_t left = uniform(K > k0 ? K - k0 : 0);  // a saturating subtraction is a vector instruction
    const uint32_t inside = KC ? left : static_cast<uint32_t>(s.n);
    uint32_t lane_off[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) lane_off[e] = c8[e] < inside ? off[e] : kOutside;
#pragma unroll
    for (int i = I0; i < I1; ++i) {
      const uint32_t q = q0 + i;
      const char* base;
      uint32_t bytes, skip = 0;
      if constexpr (KC) {
        const bool second = HALVES && q * 8 >= ROWS / 2;
        base = (second ? s.p2 : s.p) + static_cast<uint64_t>(k0) * 2;
        bytes = left ? static_cast<uint32_t>(s.n) * ld - k0 * 2 : 0;
        skip = (q * 8 - (second ? ROWS / 2 : 0)) * ld;
      } else {
        const uint32_t k = k0 + q * 2;  // even, as is K1: both rows lie in one half
        base = k < K1 ? s.p + static_cast<uint64_t>(k) * ld : s.p2 + static_cast<uint64_t>(k - K1) * ld;
        bytes = (left > q * 2 ? std::min(left - q * 2, 2u) : 0) * ld;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, bytes, 0x00020000),
                                               (__attribute__((address_space(3))) void*)(dst + q * 1024), 16,
                                               lane_off[i & 1] + skip, 0, 0, 0);
    }
  }
};

// Fragments: a lane's eight summed values (16 kk + 8 (lane / 32) ..) of row
// lane % 32 of a 32-row block.  The lane's offsets within the tile are kept in
// four registers, everything else is a constant of the read: by kk for kc (the
// chunk swizzle), by block for the other kind (the unit swizzle), whose groups of
// 16 lanes read 4 rows x 16 values each and receive them transposed.
template <bool KC>
struct Reader {
  uint32_t off[4];

  // block0: the wavefront's first block (a multiple of 4, or of the blocks it has).
  __device__ __forceinline__ Reader(int block0, int lane) {
    const int i = lane & 15, q = lane >> 4, r = lane & 31;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (KC) off[e] = (block0 * 32 + r) * 128 + (((e * 2 + (lane >> 5)) ^ ((r >> 1) & 7)) * 16);
      else off[e] = ((q >> 1) * 8 + (i >> 2)) * 512 + ((2 * ((block0 + e) ^ (i >> 2)) + (q & 1)) * 32) + (i & 3) * 8;
    }
  }

  // skip: blocks between the wavefront's first and this one beyond its number j (gate and up).
  __device__ __forceinline__ bf16x8 operator()(const char* t, int j, int kk, int skip = 0) const {
    if constexpr (KC) {
      return *reinterpret_cast<const bf16x8*>(t + off[kk] + (j + skip) * 4096);
    } else {
      typedef __attribute__((address_space(3))) bf16x4 V;
      const char* p = t + off[j] + kk * 8192;
      const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((V*)p);
      const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((V*)(p + 2048));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// A 32 x 32 block of results: lane l holds output row l % 32 and, of its 32
// columns, 8 j + 4 (l / 32) + i as v[4 j + i].  For wide stores the two halves
// of the wavefront trade: afterwards lane l holds columns 8 (2 p + l / 32) ..
// + 7, one 16-byte vector of bf16 for p = 0 and one for p = 1.
__device__ __forceinline__ void swap_halves(uint32_t& x, uint32_t& y) {
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  x = r[0];
  y = r[1];
}

// Half p of a block: its values 8 p .. 8 p + 7 of every lane, as the vector above.
__device__ __forceinline__ u32x4 pack_half(const float (&v)[8]) {
  uint32_t a0 = bf16_bits(v[0]) | (bf16_bits(v[1]) << 16);
  uint32_t a1 = bf16_bits(v[2]) | (bf16_bits(v[3]) << 16);
  uint32_t b0 = bf16_bits(v[4]) | (bf16_bits(v[5]) << 16);
  uint32_t b1 = bf16_bits(v[6]) | (bf16_bits(v[7]) << 16);
  swap_halves(a0, b0);
  swap_halves(a1, b1);
  return u32x4{a0, a1, b0, b1};
}

__device__ __forceinline__ void unpack_half(const u32x4& o, float (&v)[8]) {
  uint32_t w[4] = {o[0], o[1], o[2], o[3]};
  swap_halves(w[0], w[2]);
  swap_halves(w[1], w[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Register index against lane within each quad: afterwards v[k] of lane q is
// what v[q] of the quad's lane k was.
template <class V>
__device__ __forceinline__ void transpose_quad(V (&v)[4], int lane) {
  const auto trade = [](V& x, V& y, bool odd, auto ctrl) {  // lanes with the bit take x from the partner's y, the others y from its x
    const V px = x, py = y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t fx = __builtin_amdgcn_update_dpp(0, px[i], decltype(ctrl)::value, 0xf, 0xf, true);
      const uint32_t fy = __builtin_amdgcn_update_dpp(0, py[i], decltype(ctrl)::value, 0xf, 0xf, true);
      x[i] = odd ? fy : px[i];
      y[i] = odd ? py[i] : fx;
    }
  };
  constexpr std::integral_constant<int, 0xB1> xor1{};  // lanes 1 0 3 2
  constexpr std::integral_constant<int, 0x4E> xor2{};  // lanes 2 3 0 1
  trade(v[0], v[1], lane & 1, xor1);
  trade(v[2], v[3], lane & 1, xor1);
  trade(v[0], v[2], lane & 2, xor2);
  trade(v[1], v[3], lane & 2, xor2);
}

// Two blocks x, y as bf16 for stores of 64 contiguous bytes per quad: lane l holds, of
// block l / 32, columns 8 (l % 4) .. + 7 of row 4 (l % 32 / 4) + k as v[k].
__device__ __forceinline__ void pack_two(const f32x16& x, const f32x16& y, int lane, u32x4 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t a0 = bf16_bits(x[4 * j]) | (bf16_bits(x[4 * j + 1]) << 16);
    uint32_t a1 = bf16_bits(x[4 * j + 2]) | (bf16_bits(x[4 * j + 3]) << 16);
    uint32_t b0 = bf16_bits(y[4 * j]) | (bf16_bits(y[4 * j + 1]) << 16);
    uint32_t b1 = bf16_bits(y[4 * j + 2]) | (bf16_bits(y[4 * j + 3]) << 16);
    swap_halves(a0, b0);
    swap_halves(a1, b1);
    v[j] = u32x4{a0, a1, b0, b1};
  }
  transpose_quad(v, lane);
}

// The same in fp32, 16 of the 32 columns at a time: columns 16 p + 4 (l % 4) .. + 3.
__device__ __forceinline__ void trade_two(const f32x16& x, const f32x16& y, int p, int lane, u32x4 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a = __float_as_uint(x[8 * p + 4 * j + i]), b = __float_as_uint(y[8 * p + 4 * j + i]);
      swap_halves(a, b);
      v[2 * j][i] = a;
      v[2 * j + 1][i] = b;
    }
  transpose_quad(v, lane);
}

// bf16 store of a block: columns n0 .. n0 + 31 of the lane's row (ok: the row exists).
__device__ __forceinline__ void store_block(char* row, uint64_t n0, uint64_t N, bool ok, int lane, const f32x16& v) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = v[8 * p + e];
    const u32x4 o = pack_half(h);
    const uint64_t n = n0 + 8 * (2 * p + (lane >> 5));
    if (ok && n < N) *reinterpret_cast<u32x4*>(row + n * 2) = o;
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

// Half p of an 8-bit block, in the same places.
__device__ __forceinline__ void load_half8(const char* row, uint64_t n, uint64_t c0, int p, int lane, float (&v)[8]) {
  const float s = mx8_scale(*reinterpret_cast<const uint8_t*>(row + n + c0 / 32));
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float f[4];
    mx8_values(*reinterpret_cast<const uint32_t*>(row + c0 + 16 * p + 8 * j + 4 * (lane >> 5)), s, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * j + i] = f[i];
  }
}

// What rounding v to bf16 takes away; nothing where that is not finite.
__device__ __forceinline__ float rounded_off(float v) {
  const float d = v - __uint_as_float(bf16_bits(v) << 16);
  return fabsf(d) < __builtin_inff() ? d : 0.0f;
}

// A result and its rest's.  Where the first is infinite or NaN it stays: an infinite
// operand times a rest of 0, or of the other sign, would make NaN of an infinity.
__device__ __forceinline__ float with_rest(float v, float rest) { return fabsf(v) < __builtin_inff() ? v + rest : v; }

__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// Instruction classes of the scheduling barriers.
constexpr int kMfma = 0x8, kVmemRead = 0x20, kDsRead = 0x100;

// One matrix instruction, then R LDS reads and L loads.
template <int R, int L>
__device__ __forceinline__ void group_one() {
  __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
  if constexpr (R > 0) __builtin_amdgcn_sched_group_barrier(kDsRead, R, 0);
  if constexpr (L > 0) __builtin_amdgcn_sched_group_barrier(kVmemRead, L, 0);
}

// READS reads and LOADS loads spread evenly behind MM matrix instructions.
template <int READS, int LOADS, int MM, int... M>
__device__ __forceinline__ void group_all(std::integer_sequence<int, M...>) {
  (group_one<(READS * (M + 1)) / MM - (READS * M) / MM, (LOADS * (M + 1)) / MM - (LOADS * M) / MM>(), ...);
}

// Barrier of the workgroup that also waits for this wavefront's loads into LDS:
// behind it every wavefront's have arrived.  (A fence alone orders LDS accesses,
// and the loads count as memory accesses.)
constexpr int kLoadsDone = 0x0F70;  // vmcnt(0), the other counters free
__device__ __forceinline__ void loads_barrier() {
  __builtin_amdgcn_s_waitcnt(kLoadsDone);
  __syncthreads();
}

enum SavedKind { kNoSaved, kSaved16, kSaved8 };

// A product's tiles of TM x 256 outputs, by eight wavefronts: two along the
// rows, four along the columns, each with MB x 2 blocks of 32 x 32.  The widest
// tiles that the registers hold: each value read from LDS feeds as many matrix
// instructions as possible, and each loaded one 256 or TM results.
//
// 32768 rows over 16 experts of 4096 x 2048: gate and up 1012 us without a checkpoint
// (1.09 PFLOP/s), 1080 with one in bf16, 1070 in 8 bits; down 531 (1.04); dh 799 from
// bf16, 823 from 8 bits; dx 994 (1.11); weight gradients 503 and 971 (1.13).  Without
// its loads each takes about 80 % of that (gate and up 908 us, 453, 646, 780, 405, 745):
// a step's loads have one step to arrive, and a third LDS stage of 64 values does not fit.
// 8111 rows over 64 experts of 2048 x 1024: dh 141 us, dx 178, weight gradients
// 133 and 228, of which storing them alone takes 66 and 129.
// SAVED: the checkpoint's type (kGateUp, kDh).  F32OUT: fp32 weight gradients.
// SPLIT: rows of h are [h | rest], of g [dgate | dup | rests of both], each part
// padded to a multiple of 64 values with zeros, and row tiles half as high.
template <int KIND, int TM, int SAVED, bool F32OUT, bool SPLIT>
__global__ void __launch_bounds__(64 * kWaves, TM == 64 && !(SPLIT && (KIND == kDown || KIND == kDx)) ? 4 : 2) ffn_gemm_kernel(const GemmArgs a) {
  constexpr int WM = 2, WN = kWaves / WM;
  constexpr int MB = TM / WM / 32, NB = kTileN / WN / 32;
  constexpr bool WGRAD = KIND == kDwDown || KIND == kDwGateUp;
  constexpr bool A_KC = !WGRAD;
  constexpr bool B_KC = KIND == kGateUp || KIND == kDown;
  static_assert(!WGRAD || TM == 256, "tiles across rows are 256 wide");
  __shared__ __align__(1024) char A0[TM * 128];
  __shared__ __align__(1024) char A1[TM * 128];
  __shared__ __align__(1024) char B0[kTileN * 128];
  __shared__ __align__(1024) char B1[kTileN * 128];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / WN, wn = w % WN;
  const uint64_t H = a.H, F = a.F;
  const uint64_t FP = SPLIT ? (F + 63) & ~uint64_t(63) : F;          // a part
  const uint64_t FH = SPLIT ? 2 * FP : F, FG = (SPLIT ? 4 : 2) * FP;  // values per row of h and g
  constexpr bool PARTS = SPLIT && (KIND == kDx || WGRAD);             // sums over two parts
  constexpr bool RESTS = SPLIT && (KIND == kDown || KIND == kDx);     // rests in the tile's second half
  constexpr int ROWS = SPLIT && !WGRAD ? TM / 2 : TM;                 // rows per tile
  __shared__ f32x4 rests[RESTS ? WN : 1][RESTS ? NB * 4 : 1][kWave];
  constexpr bool A_WIDE = KIND == kDx || KIND == kDwGateUp;  // rows of 2F values
  const Loader<A_KC, TM, RESTS> load_a(KIND == kGateUp || KIND == kDh || KIND == kDwDown ? H * 2 : A_WIDE ? FG * 2 : FH * 2, w, lane);
  const Loader<B_KC, kTileN, KIND == kGateUp> load_b(KIND == kGateUp || KIND == kDx || KIND == kDwGateUp ? H * 2 : KIND == kDwDown ? FH * 2 : F * 2, w, lane);
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
    const int64_t m0 = r.m0 = static_cast<int64_t>(WGRAD ? mt : mt - sg.tile0) * ROWS;
    const int64_t n0 = r.n0 = static_cast<int64_t>(nt) * (KIND == kGateUp ? kTileN / 2 : kTileN);
    Side &A = r.A, &B = r.B;
    const uint32_t rows64 = (static_cast<uint32_t>(sg.rows) + 63) & ~63u;
    r.part = WGRAD ? rows64 : static_cast<uint32_t>(FP);
    r.sum = WGRAD ? static_cast<uint32_t>(sg.rows) : static_cast<uint32_t>(F);
    const auto left = [](int64_t most, uint64_t n) { return static_cast<int32_t>(std::min<int64_t>(most, n)); };
    if constexpr (KIND == kGateUp) {
      r.K = H;
      A = {sg.x + m0 * H * 2, nullptr, left(ROWS, sg.rows - m0)};
      B = {sg.w_gate + n0 * H * 2, sg.w_up + n0 * H * 2, left(kTileN / 2, F - n0)};
    } else if constexpr (KIND == kDown) {
      r.K = F;
      A = {a.h + (sg.row + m0) * FH * 2, a.h + ((sg.row + m0) * FH + FP) * 2, left(ROWS, sg.rows - m0)};
      B = {sg.w_down + n0 * F * 2, nullptr, left(kTileN, H - n0)};
    } else if constexpr (KIND == kDh) {
      r.K = H;
      A = {sg.dy + m0 * H * 2, nullptr, left(ROWS, sg.rows - m0)};
      B = {sg.w_down + n0 * 2, nullptr, left(kTileN, F - n0)};
    } else if constexpr (KIND == kDx) {
      r.K = 2 * FP;
      A = {a.g + (sg.row + m0) * FG * 2, a.g + ((sg.row + m0) * FG + 2 * FP) * 2, left(ROWS, sg.rows - m0)};
      B = {sg.w_gate + n0 * 2, sg.w_up + n0 * 2, left(kTileN, H - n0)};
    } else if constexpr (KIND == kDwDown) {
      r.K = SPLIT ? 2 * rows64 : sg.rows;
      A = {sg.dy + m0 * 2, nullptr, left(TM, H - m0)};
      B = {a.h + (sg.row * FH + n0) * 2, nullptr, left(kTileN, F - n0)};
      B.p2 = B.p + FP * 2;
    } else {
      r.K = SPLIT ? 2 * rows64 : sg.rows;
      A = {a.g + (sg.row * FG + m0) * 2, nullptr, left(TM, 2 * FP - m0)};
      A.p2 = A.p + FP * 4;
      B = {sg.x + n0 * 2, nullptr, left(kTileN, H - n0)};
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

  f32x16 acc[MB][NB];
  bf16x8 fa[2][MB], fb[2][NB];  // fragments of 16 summed values: those in use, and the next
  constexpr int STEPS = kTileK / 16, MM = MB * NB;
  constexpr int READS = MB * (A_KC ? 1 : 2) + NB * (B_KC ? 1 : 2);
  const Reader<A_KC> read_a(wm * MB, lane);
  const Reader<B_KC> read_b(wn * (KIND == kGateUp ? NB / 2 : NB), lane);
  auto read = [&](const char* ta, const char* tb, int kk) {
#pragma unroll
    for (int j = 0; j < NB; ++j)  // kGateUp: gate blocks, then the up blocks of the same columns
      fb[kk & 1][j] = read_b(tb, j, kk, KIND == kGateUp && j >= NB / 2 ? 4 - NB / 2 : 0);
#pragma unroll
    for (int i = 0; i < MB; ++i) fa[kk & 1][i] = read_a(ta, i, kk);
  };
  auto multiply = [&](int kk) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[kk & 1][j], fa[kk & 1][i], acc[i][j], 0, 0, 0);
  };
  constexpr uint32_t NO_K1 = ~0u;
  const uint32_t K1 = KIND == kDx ? static_cast<uint32_t>(F) : NO_K1;
  constexpr int LA = decltype(load_a)::L, LB = decltype(load_b)::L;
  // Loads of one step that run behind the barrier (the first SPLIT_A and SPLIT_B
  // instructions of each operand) and the rest, in the step that follows.
  constexpr int SPLIT_A = LA * 2 / 4, SPLIT_B = LB * 2 / 4;
  // The operand in one of the parts, of which `second` are read from p2.
  auto in_part = [](const Side& x, bool second) -> Side { return {second ? x.p2 : x.p, nullptr, x.n}; };
  auto load = [&](auto i0, auto a1, auto j0, auto b1, char* ta, char* tb, const Load& l) {
    if constexpr (PARTS) {
      const uint32_t q = uniform(l.k0 >= l.part), k = uniform(l.k0 - q * l.part);
      if constexpr (WGRAD) load_a.template run<i0.value, a1.value>(ta, in_part(l.a, KIND == kDwGateUp && !q), k, l.sum, NO_K1);
      else load_a.template run<i0.value, a1.value>(ta, l.a, l.k0, l.K, NO_K1);
      load_b.template run<j0.value, b1.value>(tb, in_part(l.b, KIND == kDx ? q : KIND == kDwDown && !q), k, l.sum, NO_K1);
    } else {
      load_a.template run<i0.value, a1.value>(ta, l.a, l.k0, l.K, NO_K1);
      load_b.template run<j0.value, b1.value>(tb, l.b, l.k0, l.K, K1);
    }
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, SPLIT_A> ca{};
  constexpr std::integral_constant<int, SPLIT_B> cb{};
  constexpr std::integral_constant<int, LA> ea{};
  constexpr std::integral_constant<int, LB> eb{};
  auto load_first = [&](char* ta, char* tb, const Load& l) { load(c0, ca, c0, cb, ta, tb, l); };
  auto load_rest = [&](char* ta, char* tb, const Load& l) { load(ca, ea, cb, eb, ta, tb, l); };
  // One step of 64 summed values from buffer (ta, tb), whose first fragments are
  // read already.  Fragments are read 16 summed values ahead of the matrix
  // instructions, across the barrier too: behind it the buffer is free, the
  // step after next is loaded into it from `src`, and the last instructions run
  // beside the other buffer's first reads.  The group barriers pin that order;
  // left alone, the compiler reads each fragment just before its use, to save
  // registers, and every read's latency shows.
  auto step = [&](char* ta, char* tb, char* na, char* nb, const Load& here, const Load& other) {
    load_rest(na, nb, other);
    read(ta, tb, 1);
    multiply(0);
    group_all<READS, LA - SPLIT_A + LB - SPLIT_B, MM>(std::make_integer_sequence<int, MM>{});
#pragma unroll
    for (int kk = 1; kk + 1 < STEPS; ++kk) {
      read(ta, tb, kk + 1);
      multiply(kk);
      group_all<READS, 0, MM>(std::make_integer_sequence<int, MM>{});
    }
    loads_barrier();
    load_first(ta, tb, here);
    read(na, nb, 0);
    multiply(STEPS - 1);
    group_all<READS, SPLIT_A + SPLIT_B, MM>(std::make_integer_sequence<int, MM>{});
  };

  // Between a weight gradient's rests and its values: an infinite operand times a rest of 0,
  // or of the other sign, leaves NaN, which an infinity of the values would not replace.
  // Any finite value does here, because that operand comes again (the median of a NaN and
  // two numbers is one of them).  1 % of a backward of 64 rows over 16 experts of
  // 2048 x 1024 (160 us, three routings).
  auto bound_rests = [&] {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = __builtin_amdgcn_fmed3f(acc[i][j][e], -__FLT_MAX__, __FLT_MAX__);
  };

  Tile cur;
  if (!advance(cur)) return;
  Load to0{cur.A, cur.B, 0, cur.K, cur.part, cur.sum}, to1{cur.A, cur.B, kTileK, cur.K, cur.part, cur.sum};  // what each buffer is filled from
  load_first(A0, B0, to0);
  load_rest(A0, B0, to0);
  load_first(A1, B1, to1);
  loads_barrier();
  read(A0, B0, 0);
  for (;;) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};
    Tile then = cur;
    const bool more = advance(then);
    const uint32_t then_K = more ? then.K : 0, then_sum = more ? then.sum : 0;
    // Two steps a turn, one from each buffer: with the buffers known at compile
    // time the reads of one need not wait for the loads into the other.  A
    // tile starts in buffer 0; its last steps already load the next tile's first
    // two, which the epilogue then hides.
    const uint32_t K = cur.K;
    uint32_t k0 = 0;
    for (; k0 + kTileK < K; k0 += 2 * kTileK) {
      const bool in0 = k0 + 2 * kTileK < K, in1 = k0 + 3 * kTileK < K;
      to0 = {pick(in0, cur.A, then.A), pick(in0, cur.B, then.B), in0 ? k0 + 2 * kTileK : 0, in0 ? K : then_K,
             in0 ? cur.part : then.part, in0 ? cur.sum : then_sum};
      if (SPLIT && WGRAD && k0 == cur.part) bound_rests();
      step(A0, B0, A1, B1, to0, to1);
      if (SPLIT && WGRAD && k0 + kTileK == cur.part) bound_rests();
      to1 = {pick(in1, cur.A, then.A), pick(in1, cur.B, then.B), in1 ? k0 + 3 * kTileK : kTileK, in1 ? K : then_K,
             in1 ? cur.part : then.part, in1 ? cur.sum : then_sum};
      step(A1, B1, A0, B0, to1, to0);
    }
    if (k0 < K || K == 0) {  // one more step, from buffer 0
      if (K <= kTileK) {
        __builtin_amdgcn_s_waitcnt(kLoadsDone);  // of what was loaded into buffer 1 for this tile: nothing, as zeros
        to1 = {then.A, then.B, kTileK, then_K, then.part, then_sum};
        load_first(A1, B1, to1);
      }
#pragma unroll
      for (int kk = 0; kk + 1 < STEPS; ++kk) {
        read(A0, B0, kk + 1);
        multiply(kk);
      }
      multiply(STEPS - 1);
      loads_barrier();
      to0 = {then.A, then.B, 0, then_K, then.part, then_sum};
      load_first(A0, B0, to0);
      load_rest(A0, B0, to0);
    }
    // The epilogue's addresses are made here: computed before the loop, as the
    // compiler would, they take the registers that the loop's own need.
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    ConstSeg& sg = *cur.sg;
    const int64_t m0 = cur.m0, n0 = cur.n0;
    if constexpr (RESTS) {
      static_assert(MB == 1, "one block of rows, one of rests");
      if (wm == 1) {
#pragma unroll
        for (int e = 0; e < NB * 4; ++e)
          rests[wn][e][lane] = f32x4{acc[0][e / 4][e % 4 * 4], acc[0][e / 4][e % 4 * 4 + 1], acc[0][e / 4][e % 4 * 4 + 2], acc[0][e / 4][e % 4 * 4 + 3]};
      }
      __syncthreads();
      if (wm == 0) {
#pragma unroll
        for (int e = 0; e < NB * 4; ++e) {
          const f32x4 q = rests[wn][e][lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[0][e / 4][e % 4 * 4 + i] = with_rest(acc[0][e / 4][e % 4 * 4 + i], q[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int64_t m = m0 + (wm * MB + i) * 32 + (lane & 31);
      if constexpr (KIND == kGateUp) {
        const bool row = m < sg.rows && (!SPLIT || wm == 0);
#pragma unroll
        for (int j = 0; j < NB / 2; ++j) {
          __builtin_amdgcn_sched_barrier(0);
          const uint64_t n = n0 + (wn * (NB / 2) + j) * 32;
          const f32x16 &gate = acc[i][j], &up = acc[i][NB / 2 + j];
          f32x16 hv;
#pragma unroll
          for (int e = 0; e < 16; ++e) hv[e] = SPLIT && n + 8 * (e / 4) >= F ? 0.0f : gate[e] * sigmoid(gate[e]) * up[e];
          char* const out_h = a.h + (sg.row + m) * FH * 2;
          store_block(out_h, n, FP, row, lane, hv);
          if constexpr (SPLIT) {
#pragma unroll
            for (int e = 0; e < 16; ++e) hv[e] = rounded_off(hv[e]);
            store_block(out_h + FP * 2, n, FP, row, lane, hv);
          }
          if constexpr (SAVED == kSaved16) {
            store_block(sg.saved + m * a.saved_row, n, F, row, lane, gate);
            store_block(sg.saved + m * a.saved_row + F * 2, n, F, row, lane, up);
          } else if constexpr (SAVED == kSaved8) {
            char* const out = sg.saved + m * a.saved_row;
            store_block8(out, 2 * F, n, row && n < F, lane, gate);
            store_block8(out, 2 * F, F + n, row && n < F, lane, up);
            if (row && n == 0 && lane < 32)  // zeros behind the scales
              for (uint64_t p = 2 * F + 2 * F / 32; p < a.saved_row; ++p) out[p] = 0;
          }
        }
      } else if constexpr (KIND == kDh) {
        const bool row = m < sg.rows && (!SPLIT || wm == 0);
        const char* in = sg.saved + static_cast<uint64_t>(std::min<int64_t>(m, sg.rows - 1)) * a.saved_row;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          __builtin_amdgcn_sched_barrier(0);
          const uint64_t n = n0 + (wn * NB + j) * 32;
          if (n >= FP) continue;
#pragma unroll
          for (int p = 0; p < 2; ++p) {  // half a block at a time, to hold few registers
            const uint64_t c = n + 8 * (2 * p + (lane >> 5));
            float gate[8], up[8], sig[8], r[8];
            if constexpr (SAVED == kSaved16) {
              const uint64_t in_c = std::min<uint64_t>(c, F - 8);
              unpack_half(*reinterpret_cast<const u32x4*>(in + in_c * 2), gate);
              unpack_half(*reinterpret_cast<const u32x4*>(in + (F + in_c) * 2), up);
            } else {
              const uint64_t in_n = std::min<uint64_t>(n, F - 32);
              load_half8(in, 2 * F, in_n, p, lane, gate);
              load_half8(in, 2 * F, F + in_n, p, lane, up);
            }
            const bool ok = row && c < FP;
            char* const out_h = a.h + (sg.row + m) * FH * 2 + c * 2;
            char* const out_g = a.g + (sg.row + m) * FG * 2 + c * 2;
            auto put = [&](char* out, uint64_t rest) {  // r, zeros in a part's padding
              const u32x4 o = pack_half(r);
              if (ok) *reinterpret_cast<u32x4*>(out) = SPLIT && c >= F ? u32x4{} : o;
              if constexpr (SPLIT) {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = rounded_off(r[e]);
                const u32x4 q = pack_half(r);
                if (ok) *reinterpret_cast<u32x4*>(out + rest * 2) = c >= F ? u32x4{} : q;
              }
            };
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              sig[e] = sigmoid(gate[e]);
              r[e] = gate[e] * sig[e] * up[e];
            }
            put(out_h, FP);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              r[e] = acc[i][j][8 * p + e] * up[e] * (sig[e] * (1.0f + gate[e] * (1.0f - sig[e])));
            put(out_g, 2 * FP);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = acc[i][j][8 * p + e] * (gate[e] * sig[e]);
            put(out_g + FP * 2, 2 * FP);
          }
        }
      } else {
        // Rows mb .. + 3 of two blocks side by side.  H and F are multiples of 8, so
        // of a weight gradient all four exist or none, and in one of its matrices.
        const int64_t mb = m0 + (wm * MB + i) * 32 + (lane & 28);
        const uint64_t M = KIND == kDwDown ? H : KIND == kDwGateUp ? FP + F : RESTS && wm == 1 ? 0 : sg.rows, N = KIND == kDwDown ? F : H;
        constexpr int ES = F32OUT ? 4 : 2;
        char* out;
        if constexpr (KIND == kDwDown) out = sg.dw_down + mb * N * ES;
        else if constexpr (KIND == kDwGateUp) out = static_cast<uint64_t>(mb) < FP ? sg.dw_gate + mb * N * ES : sg.dw_up + (mb - static_cast<int64_t>(FP)) * N * ES;
        else out = sg.y + mb * N * ES;
#pragma unroll
        for (int p = 0; p < (F32OUT ? 2 : 1); ++p) {
          __builtin_amdgcn_sched_barrier(0);
          const uint64_t n = n0 + (wn * NB + (lane >> 5)) * 32 + (F32OUT ? 16 * p + 4 * (lane & 3) : 8 * (lane & 3));
          u32x4 v[4];
          if constexpr (F32OUT) trade_two(acc[i][0], acc[i][1], p, lane, v);
          else pack_two(acc[i][0], acc[i][1], lane, v);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (static_cast<uint64_t>(mb + (WGRAD ? 0 : k)) < M && n < N && !(SPLIT && KIND == kDwGateUp && static_cast<uint64_t>(mb) >= F && static_cast<uint64_t>(mb) < FP)) *reinterpret_cast<u32x4*>(out + (k * N + n) * ES) = v[k];
        }
      }
    }
    // Every way to the next tile waits here, the last one's too.  Waiting only
    // after an odd number of steps would be enough, but the compiler then sees a
    // way to the loop with buffer 0 still loading and waits for every load at the
    // loop's head (3 to 5 % of a large product).
    loads_barrier();
    if (!more) break;
    read(A0, B0, 0);
    cur = then;
  }
}

// ------------------------------------------------------------------ few rows
//
// Serving: a handful of rows per expert, where a product is one pass over the
// weights.  A wavefront owns 16 output columns of one expert (of both matrices
// for gate and up) and a share of the summed index: it streams the weights
// straight into the matrix instructions' registers (16 rows x 32 summed values
// each, 64 bytes a row and instruction, kFewLoads KiB in flight).  The
// workgroup's eight wavefronts are `shares` shares of 8 / shares column groups;
// shares are added through LDS in a fixed order.  h is kept as two bf16 values here
// too: the down product takes eight rows at a time, with their rests as the other
// eight columns of the matrix instructions.  The expert's rows are found
// from the split table by the workgroup itself, so the whole forward is two
// launches.  HBM bytes bound it: two experts of 4096 x 11008 with a row each, gate
// and up 84 us (4.3 TB/s), down 44 us (4.1 TB/s).

constexpr int kFewWaves = 8;
constexpr int kFewLoads = 8;  // weight vectors in flight per lane

template <int P>
struct FewArgs {
  const char* x[P];        // rows that gate and up multiply
  const char* wa[P];
  const char* wb[P];       // up; unused by down
  char* y[P];
  int64_t rows[P];
  int64_t base[P];         // rows of the ranks before
  const int64_t* splits;
  char* h;
  uint64_t K, n;           // summed values, output columns
  uint32_t N, E, tiles;    // column tiles per expert: at most 2^16 of at most kFewSegs experts, 2^31 work items
  uint32_t shares;         // of the summed index: 1, 2, 4 or 8
};

__device__ __forceinline__ int64_t wave_sum64(int64_t x) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

template <bool GATE_UP, int P>
__global__ void __launch_bounds__(64 * kFewWaves) ffn_few_kernel(const FewArgs<P> a) {
  constexpr int U = GATE_UP ? kFewLoads / 2 : kFewLoads;
  constexpr int TURN = GATE_UP ? 16 : 8;  // rows at a time; down: beside their rests
  __shared__ f32x4 part[kFewWaves][GATE_UP ? 2 : 1][kWave];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t share = w % a.shares, group = w / a.shares, groups = kFewWaves / a.shares;
  const uint32_t seg = blockIdx.x / a.tiles;
  const uint32_t d = seg / a.E, e = seg - d * a.E;
  int64_t before = 0, count = 0;
  for (uint32_t i = lane; i < (e + 1) * a.N; i += kWave) {
    const uint32_t q = i / a.N, s = i - q * a.N;
    const int64_t v = a.splits[(static_cast<uint64_t>(s) * a.N + d) * a.E + q];
    const int64_t c = min(max(v, int64_t(0)), a.rows[d]);
    if (q < e) before += c;
    else count += c;
  }
  before = wave_sum64(before);
  count = wave_sum64(count);
  const int64_t start = min(before, a.rows[d]);
  const int64_t rows = min(before + count, a.rows[d]) - start;
  const uint64_t n0 = static_cast<uint64_t>((blockIdx.x - seg * a.tiles) * groups + group) * 16;
  const uint64_t col = min(n0 + (lane & 15), a.n - 1);  // past the last: the last again, not stored
  const uint64_t w0 = (static_cast<uint64_t>(e) * a.n + col) * a.K * 2;
  const char* const wa = a.wa[d] + w0;
  const char* const wb = GATE_UP ? a.wb[d] + w0 : nullptr;
  for (int64_t m0 = 0; m0 < rows; m0 += TURN) {
    const int64_t m = min(m0 + lane % TURN, rows - 1);
    const char* const x = GATE_UP ? a.x[d] + (start + m) * a.K * 2 : a.h + ((a.base[d] + start + m) * 2 + (lane >> 3 & 1)) * a.K * 2;
    f32x4 ga{}, ua{};
    for (uint64_t k0 = static_cast<uint64_t>(share) * 32 * U; k0 < a.K; k0 += 32 * U * a.shares) {
      u32x4 va[U], vb[U], vx[U];  // vb: up
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint64_t k = k0 + i * 32 + (lane >> 4) * 8;
        const uint64_t c = k < a.K ? k * 2 : 0;  // clamped: no exec-masked load
        va[i] = ld16(wa + c);
        if constexpr (GATE_UP) vb[i] = ld16(wb + c);
        vx[i] = *reinterpret_cast<const u32x4*>(x + c);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (k0 + i * 32 + (lane >> 4) * 8 >= a.K) {  // past the end: zeros on both sides
          va[i] = u32x4{};
          if constexpr (GATE_UP) vb[i] = u32x4{};
          vx[i] = u32x4{};
        }
        ga = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, va[i]), __builtin_bit_cast(bf16x8, vx[i]), ga, 0, 0, 0);
        if constexpr (GATE_UP)
          ua = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, vb[i]), __builtin_bit_cast(bf16x8, vx[i]), ua, 0, 0, 0);
      }
    }
    part[w][0][lane] = ga;
    if constexpr (GATE_UP) part[w][1][lane] = ua;
    __syncthreads();
    if (share == 0) {
      for (uint32_t q = 1; q < a.shares; ++q) {
        ga += part[w + q][0][lane];
        if constexpr (GATE_UP) ua += part[w + q][1][lane];
      }
      if constexpr (!GATE_UP) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ga[i] = with_rest(ga[i], __shfl_xor(ga[i], 8));
      }
      // lane l: row m0 + l % 16 (down: and its rest, l % 8), columns n0 + 4 (l / 16) .. + 3
      const uint64_t n = n0 + 4 * (lane >> 4);
      if (m0 + lane % TURN < rows && (lane & 15) < TURN && n < a.n) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = GATE_UP ? ga[i] * sigmoid(ga[i]) * ua[i] : ga[i];
        char* const out = GATE_UP ? a.h + (a.base[d] + start + m) * a.n * 4 : a.y[d] + (start + m) * a.n * 2;
        *reinterpret_cast<u32x2*>(out + n * 2) =
            u32x2{bf16_bits(v[0]) | (bf16_bits(v[1]) << 16), bf16_bits(v[2]) | (bf16_bits(v[3]) << 16)};
        if constexpr (GATE_UP) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = rounded_off(v[i]);
          *reinterpret_cast<u32x2*>(out + (a.n + n) * 2) =
              u32x2{bf16_bits(v[0]) | (bf16_bits(v[1]) << 16), bf16_bits(v[2]) | (bf16_bits(v[3]) << 16)};
        }
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host side

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
  const uint64_t grid = grid_for(a.mtiles * a.ntiles, g.tile_rows > 64 || (g.split && (KIND == kDown || KIND == kDx)) ? 1 : 2);
  if (g.split) return launch(ffn_gemm_kernel<KIND, 64, SAVED, false, true>, a, grid, 64 * kWaves, stream);
  if (g.tile_rows == 256) return launch(ffn_gemm_kernel<KIND, 256, SAVED, false, false>, a, grid, 64 * kWaves, stream);
  if (g.tile_rows == 128) return launch(ffn_gemm_kernel<KIND, 128, SAVED, false, false>, a, grid, 64 * kWaves, stream);
  return launch(ffn_gemm_kernel<KIND, 64, SAVED, false, false>, a, grid, 64 * kWaves, stream);
}

template <int KIND, bool SPLIT>
gc_status weight_product(GemmArgs a, uint64_t M, uint64_t N, bool f32, hipStream_t stream) {
  a.mtiles = ceil_div(M, 256);
  a.ntiles = ceil_div(N, kTileN);
  const uint64_t grid = grid_for(a.mtiles * a.ntiles * a.segs_n, 1);
  if (f32) return launch(ffn_gemm_kernel<KIND, 256, kNoSaved, true, SPLIT>, a, grid, 64 * kWaves, stream);
  return launch(ffn_gemm_kernel<KIND, 256, kNoSaved, false, SPLIT>, a, grid, 64 * kWaves, stream);
}

template <bool SPLIT>
gc_status weight_gradients(const gci::FfnCall& c, const GemmArgs& a) {
  const gc_status st = weight_product<kDwDown, SPLIT>(a, c.hidden, c.inter, c.dw_t == GC_FP32, c.stream);
  if (st != GC_OK) return st;
  const uint64_t part = SPLIT ? (c.inter + 63) & ~uint64_t(63) : c.inter;
  return weight_product<kDwGateUp, SPLIT>(a, 2 * part, c.hidden, c.dw_t == GC_FP32, c.stream);
}

// Shares of the summed index: about four turns of a wavefront's loads each, so
// that short ones do not leave a workgroup less work than finding its rows, and
// long ones are spread over all of its wavefronts.
template <class A>
void split_few(A& a, int unroll) {
  a.shares = 1;
  while (a.shares < kFewWaves && a.K > static_cast<uint64_t>(32 * unroll * 4) * a.shares) a.shares *= 2;
  a.tiles = static_cast<uint32_t>(ceil_div(a.n, 16 * (kFewWaves / a.shares)));
}

template <int P>
gc_status forward_few(const gci::FfnCall& c, const gci::FfnGeom& g) {
  FewArgs<P> a{};
  char* const base = static_cast<char*>(c.scratch);
  int64_t run = 0;
  for (int d = 0; d < c.nranks; ++d) {
    a.x[d] = c.x_t == GC_MX8 ? base + g.x + run * c.hidden * 2 : static_cast<const char*>(c.x[d]);
    a.wa[d] = static_cast<const char*>(c.w_gate[d]);
    a.wb[d] = static_cast<const char*>(c.w_up[d]);
    a.y[d] = static_cast<char*>(c.y[d]);
    a.rows[d] = c.rows[d];
    a.base[d] = run;
    run += c.rows[d];
  }
  a.splits = c.splits;
  a.h = base + g.h;
  a.K = c.hidden;
  a.n = c.inter;
  a.N = c.nranks;
  a.E = c.experts_per_rank;
  split_few(a, kFewLoads / 2);
  const gc_status st = launch(ffn_few_kernel<true, P>, a, static_cast<uint64_t>(g.segs) * a.tiles, 64 * kFewWaves, c.stream);
  if (st != GC_OK) return st;
  for (int d = 0; d < c.nranks; ++d) a.wa[d] = static_cast<const char*>(c.w_down[d]);
  a.K = c.inter;
  a.n = c.hidden;
  split_few(a, kFewLoads);
  return launch(ffn_few_kernel<false, P>, a, static_cast<uint64_t>(g.segs) * a.tiles, 64 * kFewWaves, c.stream);
}

}  // namespace

namespace gci {

gc_status launch_moe_ffn(const FfnCall& c) {
  const FfnGeom g = ffn_geom(c.rows, c.nranks, c.experts_per_rank, c.hidden, c.inter, c.x_t, false);
  if (g.rows == 0) return GC_OK;
  if (!c.saved && g.few) {
    const gc_status st = decode_x(c, g);
    if (st != GC_OK) return st;
    return c.nranks <= 8 ? forward_few<8>(c, g) : forward_few<64>(c, g);
  }
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
  return g.split ? weight_gradients<true>(c, a) : weight_gradients<false>(c, a);
}

}  // namespace gci
