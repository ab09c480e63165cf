// MI355X (gfx950, CDNA4) kernels for the experts that stand between dispatch
// and combine, behind the C ABI declared in include/moe_route.h: the gated
// block's two projections, the matrix product with its epilogue, their
// gradients, and combine's gradient.
//
// The rows are dispatch's: expert-major and packed, expert e's rows in
// [expert_offsets[e], expert_offsets[e+1]).  The offsets stay on the device,
// so every launch is sized from the number of rows and experts alone and a
// block finds its expert by a prefix sum over the experts' tile counts.
//
// Every product is D[m][n] = sum_k Q[m][k] * P[n][k] with Q the side of the
// rows of the output and P the side of its contiguous index:
//
//   forward       m = row, n = output feature, k = input feature
//   data gradient m = row, n = input feature,  k = output feature
//   weight grad   m = output feature, n = input feature, k = row
//
// P is the matrix instruction's first operand, so that a lane ends up with
// consecutive n of one m and stores them together.

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "moe_route.h"

namespace {

constexpr int kWave = 64;
constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr int64_t kMaxPairs = (int64_t(1) << 31) - 1;
constexpr int kMaxFeatures = 1 << 20;
constexpr int64_t kMaxBlocks = int64_t(1) << 20;  // blocks loop over tiles past this
constexpr int64_t kMaxTiles = (int64_t(1) << 31) - 1;
constexpr int kCus = 256;  // blocks of a kernel that goes through its tiles in one sequence

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int lane_id() { return threadIdx.x & (kWave - 1); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));  // nearest even
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------

// They run on every value of a product's tile, so they are built on the hardware's exp2 and reciprocal
// (1 ulp each).  The argument of exp2 is rounded in fp32, so the relative error grows with |z|, to
// 2^-18 |z| at most: far below half a step of bf16, as which the result is stored.

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// 1 / (1 + exp(-z)); exp2 overflows to infinity for z < -88, which gives 0.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// Phi(z), the normal distribution function, and exp(-z^2 / 2).  The tail Phi(-x), x >= 0, is
// exp(-x^2 / 2) t P(t) with t = 1 / (1 + 0.3 x): the factor t P(t) falls like 1 / x and is smooth in
// t, so that P of degree 7, fitted here to a least largest relative error over 0 <= x <= 14, holds it
// to 1.5e-7 (4.7e-7 evaluated in fp32).  The left tail keeps its relative precision, where 1 + erf
// would cancel.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float x = __builtin_fabsf(z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, x, 1.0f));
  e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * (z * z));
  float p = 0.0356763f;
  p = __builtin_fmaf(p, t, -0.15720925f);
  p = __builtin_fmaf(p, t, 0.20636382f);
  p = __builtin_fmaf(p, t, -0.05369288f);
  p = __builtin_fmaf(p, t, 0.12856639f);
  p = __builtin_fmaf(p, t, 0.09991208f);
  p = __builtin_fmaf(p, t, 0.12075418f);
  p = __builtin_fmaf(p, t, 0.11962928f);
  const float tail = e * (p * t);
  return z < 0.f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  float e;
  if constexpr (ACT == MOE_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == MOE_ACT_GELU) return z * normal_cdf(z, e);
  if constexpr (ACT == MOE_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays one
  return z;
}

// d act / dz (relu's is 0 at 0).
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  float e;
  if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoid(z);
    return s * (1.f + z * (1.f - s));
  }
  if constexpr (ACT == MOE_ACT_GELU) {
    const float phi = normal_cdf(z, e);
    return __builtin_fmaf(z * e, kInvSqrt2Pi, phi);
  }
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  return 1.f;
}

// f(integral_constant<int, act>): one branch in front of a loop over rows, whose code is then one
// short piece.  With the branch inside, a tile's epilogue took 7 us longer, mostly to fetch it.
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F f) {
  if (act == MOE_ACT_SILU)
    f(std::integral_constant<int, MOE_ACT_SILU>{});
  else if (act == MOE_ACT_GELU)
    f(std::integral_constant<int, MOE_ACT_GELU>{});
  else if (act == MOE_ACT_RELU)
    f(std::integral_constant<int, MOE_ACT_RELU>{});
  else
    f(std::integral_constant<int, MOE_ACT_NONE>{});
}

// ---------------------------------------------------------------------------
// an expert's rows, and which tile of which expert a block computes
// ---------------------------------------------------------------------------

// Rows [lo, lo + n) of expert e.  Offsets outside [0, rows] or out of order
// are held to the buffer, so that no access leaves it.
__device__ __forceinline__ void expert_rows(const int32_t* off, int e, int64_t rows, int64_t& lo,
                                            int64_t& n) {
  int64_t a = off[e], b = off[e + 1];
  a = a < 0 ? 0 : (a > rows ? rows : a);
  b = b < a ? a : (b > rows ? rows : b);
  lo = a;
  n = b - a;
}

// How the n rows of an expert are cut into tiles of at most BM rows, BM = FULL or FULL + 32: `count`
// tiles of `height` rows, a multiple of 32 (the last may be shorter).  Tiles of FULL rows, unless these
// leave a last one that is at most half full where FULL + 32 rows need one tile less: a short tile
// costs far more than its share, as it waits for the same weights.  Then the rows are spread evenly.
template <int FULL, int BM>
__device__ __forceinline__ void cut_rows(uint32_t n, int& count, int& height) {
  uint32_t c = (n + FULL - 1) / FULL;
  height = FULL;
  if (BM > FULL) {
    const uint32_t fewer = (n + BM - 1) / BM;
    if (fewer < c && n - (c - 1) * FULL <= FULL / 2) c = fewer;
    const uint32_t h = c > 1 ? (n + c - 1) / c : n;
    height = int((h + 31) / 32 * 32);
    if (c > 1) c = (n + height - 1) / uint32_t(height);
  }
  count = int(c);
}

// A value every lane of the wave has, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return int64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(v)))) |
         int64_t(__builtin_amdgcn_readfirstlane(int(v >> 32))) << 32;
}

// The same for an expert that is the same for the whole wave: through the scalar cache, whose loads
// are waited for apart from the vector loads and stores under way.
__device__ __forceinline__ void expert_rows_scalar(const int32_t* off, int e, int64_t rows,
                                                   int64_t& lo, int64_t& n) {
  typedef const __attribute__((address_space(4))) int32_t* Scalar;
  const Scalar o = (Scalar)(off);
  e = __builtin_amdgcn_readfirstlane(e);
  int64_t a = o[e], b = o[e + 1];
  a = a < 0 ? 0 : (a > rows ? rows : a);
  b = b < a ? a : (b > rows ? rows : b);
  lo = a;
  n = b - a;
}

struct Tile {
  int e;         // expert, or -1 past the last tile
  int64_t row0;  // first row
  int rows;      // rows of this tile (1 .. BM)
  int nt;        // column tile
};

// Blocks are handed to the 8 XCDs in turn, and each XCD has an L2 of its own.
// So that the tiles an XCD works on at one time share their operands, tile
// numbers go to the XCDs in runs of 32 (its CUs), and what is left of `total`
// after the last round of such runs in runs half as long, and so on: a bijection
// on [0, total).  From `total` on the number is returned as it is.
constexpr uint32_t kXcds = 8;

__device__ __forceinline__ uint32_t xcd_order(uint32_t id, uint32_t total) {
  uint32_t base = 0;
#pragma unroll
  for (uint32_t run = 32; run >= 1; run >>= 1) {
    const uint32_t span = (total - base) / (kXcds * run) * (kXcds * run);
    if (id < base + span) {
      const uint32_t i = id - base, j = i / kXcds;
      return base + (j / run * kXcds + i % kXcds) * run + j % run;
    }
    base += span;
  }
  return id;
}

// Tile `local` of a grid of mt x nt tiles: strips of 8 row tiles, inside a strip
// the row tile first, so that 32 neighbours read 8 + 4 strips of the operands.
__device__ __forceinline__ void grid_order(uint32_t local, uint32_t mt, uint32_t nt, int& m,
                                           int& n) {
  const uint32_t g = local / (8 * nt), rem = local - g * 8 * nt;
  const uint32_t gm = mt - g * 8 < 8 ? mt - g * 8 : 8;
  n = int(rem / gm);
  m = int(g * 8 + rem % gm);
}

// Inclusive prefix sum over the 64 lanes: four shifts inside each 16-lane row, then each row's total
// into the rows above it.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_zero(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_prefix(int v) {
  v += dpp_or_zero<0x111, 0xF>(v);  // row_shr:1
  v += dpp_or_zero<0x112, 0xF>(v);
  v += dpp_or_zero<0x114, 0xF>(v);
  v += dpp_or_zero<0x118, 0xF>(v);
  v += dpp_or_zero<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v += dpp_or_zero<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return v;
}

// The tile of block number `id`.  Every thread of the block calls it.  Each thread counts the row
// tiles of `kPer` experts; the one that holds the tile writes it down.  The host refuses more than 2^31 - 1 tiles.
template <int FULL, int BM, int THREADS>
__device__ Tile find_tile(const int32_t* off, int E, int64_t rows, int ncol, uint32_t id) {
  constexpr int kPer = kMaxE / THREADS, kWaves = THREADS / kWave;
  __shared__ int s_wave[kWaves];
  __shared__ Tile s_tile;
  int64_t lo[kPer];
  int n[kPer], mt[kPer], height[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    int64_t cnt = 0;
    lo[i] = 0;
    if (e < E) expert_rows(off, e, rows, lo[i], cnt);
    n[i] = int(cnt);
    cut_rows<FULL, BM>(uint32_t(cnt), mt[i], height[i]);
    mine += mt[i];
  }
  const int incl = wave_prefix(mine);
  const int w = threadIdx.x / kWave;
  if (threadIdx.x == 0) s_tile.e = -1;
  if (lane_id() == kWave - 1) s_wave[w] = incl;
  __syncthreads();
  int pre = incl - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const int v = s_wave[i];
    if (i < w) pre += v;
    total += v;
  }
  const uint32_t tiles = uint32_t(__builtin_amdgcn_readfirstlane(total)) * uint32_t(ncol);
  if (id < tiles) {
    int local = int(xcd_order(id, tiles)) - pre * ncol;
    if (local >= 0 && local < mine * ncol) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (local >= 0 && local < mt[i] * ncol) {
          int m, c;
          grid_order(local, mt[i], ncol, m, c);
          const int left = n[i] - m * height[i];
          s_tile.e = threadIdx.x * kPer + i;
          s_tile.row0 = lo[i] + m * height[i];
          s_tile.rows = left < height[i] ? left : height[i];
          s_tile.nt = c;
        }
        local -= mt[i] * ncol;
      }
    }
  }
  __syncthreads();
  Tile t = s_tile;
  __syncthreads();  // s_tile and s_wave may be written again
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  t.nt = __builtin_amdgcn_readfirstlane(t.nt);
  t.row0 = uniform(t.row0);
  return t;
}

// ---------------------------------------------------------------------------
// operand tiles in LDS
// ---------------------------------------------------------------------------
//
// A stage holds 64 values of k for each side.  It is filled by buffer loads
// that write LDS directly, 16 bytes a lane: the 64 lanes of one load fill 1 KiB
// of consecutive LDS, so the order of chunks inside a tile is chosen by which
// chunk each lane reads.  A load past the resource's end writes zeros, which is
// how rows and k outside the operand enter the product as zeros on both sides
// (a 0 against another expert's NaN would not do).
//
//   k contiguous (KC): LDS row = position, 128 bytes = 64 k = 8 chunks; chunk c
//     of row r sits in slot c ^ (r & 7), so that lanes that a 128-bit read serves
//     at once, rows apart by 128 bytes, find different banks.
//   position contiguous: LDS row = k, R positions; read transposed
//     (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 values and each receives
//     one column).  32 lanes are served at once, 8 rows; chunk c of row k sits
//     in slot c ^ (2 (k & 3) + (k & 8)), which puts their 8 pieces of 32 bytes
//     in different banks of the 64.

constexpr int kBK = 64;
constexpr uint32_t kOutside = 0x80000000u;  // past every resource (at most 2^30 bytes)

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int wave_id() {
  return __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
}

__device__ __forceinline__ i32x4 resource(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return i32x4{__builtin_amdgcn_readfirstlane(int(b)),
               __builtin_amdgcn_readfirstlane(int(b >> 32)),
               __builtin_amdgcn_readfirstlane(int(bytes)), 0x00020000};
}

// 16 bytes a lane from base + voff + soff to LDS lds + 16 * lane.  The load has no
// register output; `stage_ready` waits for it.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t voff, i32x4 rsrc, int soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff));
}

// The same for data that no other block reads: it is not kept in the caches.
__device__ __forceinline__ void load_once_to_lds(uint32_t lds, uint32_t voff, i32x4 rsrc, int soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen nt lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff));
}

// All but the newest N loads of this wave have arrived and its LDS reads are
// done; then the same holds for every wave of the block.
template <int N>
__device__ __forceinline__ void stage_ready() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) const void*)p));
}

// One side of R positions, loaded by W waves.
template <bool KC_, int R, int W, bool TWO = false, bool ONCE = false>
struct Side {
  static constexpr bool KC = KC_;
  static constexpr int kBytes = R * kBK * 2;
  static constexpr int kLoads = kBytes / 1024 / W;  // a wave's loads per stage
  static constexpr int kKRows = 512 / R;            // !KC: values of k in one load
  static constexpr int kRow = R * 2;                // !KC: bytes of an LDS row

  uint32_t voff;  // this lane's place in load 0; load J goes by a resource that starts `ahead<J>` further
  i32x4 rsrc, rsrc2;  // KC: of the positions whose bit 5 is clear / set (they differ if gated)
  const uint16_t* base;
  int64_t ld;
  int whole, tail;  // stages full of k, and the k left for one more
  uint32_t stage_bytes;
  uint32_t skip;  // !KC: bytes in front of the first column
  int kc;         // KC: this lane's k in the stage

  // KC: `first` points at position 0, k 0, and `valid` rows from there exist.  TWO: positions
  // 64 s + j are row 32 s + j behind `first` (j < 32) or row 32 s + j - 32 behind `second`.
  __device__ __forceinline__ void init_kc(const uint16_t* first, const uint16_t* second,
                                          int64_t ld_, int64_t K_, int64_t valid) {
    ld = ld_;
    whole = __builtin_amdgcn_readfirstlane(int(K_ / kBK));
    tail = __builtin_amdgcn_readfirstlane(int(K_ % kBK));
    const uint32_t bytes = valid <= 0 ? 0u : uint32_t(valid < R ? valid : R) * uint32_t(ld * 2);
    rsrc = resource(first, bytes);
    rsrc2 = TWO ? resource(second, bytes) : rsrc;
    const int l = lane_id(), c = (l % 8) ^ (l / 8);
    kc = c * 8;
    const int r = wave_id() * 8 + l / 8;
    voff = uint32_t(TWO ? r % 32 : r) * uint32_t(ld * 2) + c * 16;
  }

  // !KC: `first` points at k 0 of the first position, which is column `col` of its row.
  __device__ __forceinline__ void init_mc(const uint16_t* first, int64_t ld_, int64_t K_, int col) {
    base = first;
    ld = ld_;
    whole = __builtin_amdgcn_readfirstlane(int(K_ / kBK));
    tail = __builtin_amdgcn_readfirstlane(int(K_ % kBK));
    skip = __builtin_amdgcn_readfirstlane(col * 2);
    stage_bytes = kBK * uint32_t(ld * 2) - skip;
    const int l = lane_id(), k = wave_id() * kKRows + l / (R / 8);
    voff = uint32_t(k) * uint32_t(ld * 2) + ((l % (R / 8)) ^ (((k & 3) << 1) | (k & 8))) * 16;
  }

  // Rows of the operand between load 0 and load J of a wave.
  template <int J>
  static constexpr int kAhead = !KC ? J * W * kKRows : TWO ? J * W * 8 / 64 * 32 : J * W * 8;
  // The resource of load J: what is behind the rows in front of it.
  template <int J>
  __device__ __forceinline__ i32x4 ahead(i32x4 r) const {
    if constexpr (kAhead<J> == 0) return r;
    const uint32_t by = kAhead<J> * uint32_t(ld * 2);
    const uint64_t b = (uint64_t(uint32_t(r[1])) << 32 | uint32_t(r[0])) + by;
    const int left = r[2] - int(by);
    return i32x4{int(uint32_t(b)), int(uint32_t(b >> 32)), left > 0 ? left : 0, r[3]};
  }

  // The resource that a stage's loads go through: the k of stage `it` (!KC), or the side's own.
  template <bool WHOLE>
  __device__ __forceinline__ i32x4 stage_resource(int it) const {
    if constexpr (KC) return rsrc;
    const uint32_t n = WHOLE || it < whole ? stage_bytes
                       : it == whole && tail > 0 ? uint32_t(tail) * uint32_t(ld * 2) - skip : 0u;
    return resource(base + (WHOLE || it <= whole ? int64_t(it) * kBK * ld : 0), n);
  }

  static __device__ __forceinline__ void bring(uint32_t lds, uint32_t v, i32x4 r, int soff) {
    if constexpr (ONCE)
      load_once_to_lds(lds, v, r, soff);
    else
      load_to_lds(lds, v, r, soff);
  }

  // Start this wave's load J of the stage at `lds` (this wave's first KiB of the side there), which
  // takes k in [64 it, 64 it + 64).  WHOLE: all of these exist.
  template <int J, bool WHOLE>
  __device__ __forceinline__ void issue(uint32_t lds, i32x4 r, int it) const {
    if constexpr (!KC) {
      bring(lds + J * W * 1024, voff, ahead<J>(r), 0);
    } else {
      if (TWO && (W == 8 ? wave_id() >> 2 : J * W >> 2 & 1)) r = rsrc2;
      const bool some = WHOLE || it <= whole;
      const uint32_t v = WHOLE || it < whole || (it == whole && kc < tail) ? voff : kOutside;
      bring(lds + J * W * 1024, v, ahead<J>(r), some ? it * (kBK * 2) : 0);
    }
  }

  // Where this lane reads in the side's part of a stage: KC, the address of fragment 0 in each half
  // stage; else that of each of the first 128 / STEP fragments (256 bytes on, the swizzle is the same).
  // Fragment f is positions row0 + f * STEP .. + 15, f < FRAGS.
  template <int STEP, int FRAGS>
  static constexpr int kBases = KC ? 2 : FRAGS < 128 / STEP ? FRAGS : 128 / STEP;
  template <int STEP, int N>
  static __device__ __forceinline__ void read_bases(uint32_t (&at)[N], uint32_t lds, int row0) {
    const int l = lane_id(), i = l % 16, q = l / 16;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (KC) {
        at[u] = lds + (row0 + i) * 128 + (((u * 4 + q) ^ (i & 7)) * 16);
      } else {
        const int chunk = (row0 + u * STEP) / 8 + (i % 4) / 2;
        at[u] = lds + (q * 8 + i / 4) * kRow +
                ((chunk ^ (((i / 4) << 1) | ((q & 1) << 3))) * 16) + (i & 1) * 8;
      }
    }
  }

  // Fragment F of half stage SUB, 8 values of k per lane, of the stage `at` was moved to.
  template <int F, int STEP, int SUB, int N>
  static __device__ __forceinline__ bf16x8 read(const uint32_t (&at)[N]) {
    typedef __attribute__((address_space(3))) const bf16x8* Frag;
    typedef __attribute__((address_space(3))) s16x4* Tr;
    if constexpr (KC) {
      return *reinterpret_cast<Frag>(at[SUB] + F * STEP * 128);
    } else {
      constexpr int kPer = 128 / STEP;
      const uint32_t p = at[F % kPer] + (F / kPer * 256 + SUB * 32 * kRow);
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<Tr>(p));
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<Tr>(p + 4 * kRow));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// f(integral_constant<int, 0>) .. f(integral_constant<int, N - 1>)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// The tile shape: up to BM x BN outputs (rows are cut by FULL, see cut_rows) by WM x WN waves.  A wave's
// row fragment i covers rows 16 (i * WM + wave row), so that a short tile loads every wave alike.
template <int FULL_, int BM_, int BN_, int WM_, int WN_, int LDS_, bool ONCE = false>
struct Shape {
  static constexpr bool kOnce = ONCE;  // the weights are read by one block each
  static constexpr int FULL = FULL_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, kLds = LDS_;
  static constexpr int W = WM * WN, kThreads = W * kWave;
  static constexpr int kWaveN = BN / WN, MR = BM / WM / 16, NR = kWaveN / 16;
  // Rows that one load of every wave brings, and the rows a stage holds for MREP row fragments.
  static constexpr int kLoadRows = W * 8;
  template <int MREP>
  static constexpr int kRows = (MREP * 16 * WM + kLoadRows - 1) / kLoadRows * kLoadRows;
  // As many stages as fit, 4 at most.
  template <int BYTES>
  static constexpr int kStages = kLds / BYTES < 4 ? kLds / BYTES : 4;
};

// A value that the compiler takes as it finds it: what is added to it stays in the offsets of the
// instructions that use it.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
__device__ __forceinline__ int opaque_scalar(int v) {
  asm volatile("" : "+s"(v));
  return v;
}

// The product of a tile: acc[a][u] is positions 16 u + 4 (lane / 16) .. + 3 of the wave's, against row
// lane % 16 of its row fragment a, for MREP row fragments.
//
// A step takes one stage in two halves of MREP groups of NR matrix instructions.  While a half is
// computed the next half's fragments are read, each row fragment into the registers that the group
// before has just used.  The second half reads from the next stage: kHead groups into it stands the
// barrier that hands that stage over, so that these groups cover the end of the reads and the
// barrier.  With it the current stage has been read by all, and the loads of the stage ST further on
// go into its place, spread over the rest of the half: issued together they hold up every wave for
// as long as the CU's one address unit takes for all of them.
//
// The stages of one tile may be followed by those of another: `run` ends with the next tile's first
// ST stages under way and the first half of its first stage in registers.
template <typename S, int MREP, typename PS, typename QS>
struct Pipe {
  static constexpr int kStage = PS::kBytes + QS::kBytes, ST = S::template kStages<kStage>;
  static_assert(ST >= 2, "one stage is computed while the next arrives");
  static constexpr int kLoads = PS::kLoads + QS::kLoads;
  static constexpr int kHead = MREP >= 4 ? 2 : 1, kStep = 16 * S::WM;

  static constexpr int kPB = PS::template kBases<16, S::NR>, kQB = QS::template kBases<kStep, MREP>;

  uint32_t pat[kPB], qat[kQB];  // where this lane reads, in the stage being read
  int dest, cur;
  bf16x8 p[2][S::NR], q[MREP];

  __device__ __forceinline__ void move_by(int bytes) {
#pragma unroll
    for (int u = 0; u < kPB; ++u) pat[u] = opaque(pat[u] + bytes);
#pragma unroll
    for (int u = 0; u < kQB; ++u) qat[u] = opaque(qat[u] + bytes);
  }
  template <int J, bool WHOLE>
  __device__ __forceinline__ void load(const PS& P, const QS& Q, int stage, int it, i32x4 pr,
                                       i32x4 qr) {
    if constexpr (J < PS::kLoads)
      P.template issue<J, WHOLE>(dest + stage * kStage, pr, it);
    else
      Q.template issue<J - PS::kLoads, WHOLE>(dest + stage * kStage + PS::kBytes, qr, it);
  }
  // One of the NR + MREP fragments of half SUB, in the order of use.
  template <int SUB, int I>
  __device__ __forceinline__ void read() {
    if constexpr (I == 0)
      q[0] = QS::template read<0, kStep, SUB>(qat);
    else if constexpr (I <= S::NR)
      p[SUB][I - 1] = PS::template read<I - 1, 16, SUB>(pat);
    else
      q[I - S::NR] = QS::template read<I - S::NR, kStep, SUB>(qat);
  }
  // Reads after group A of a half whose first FROM groups read nothing: one row fragment for each
  // group passed, and P's fragments with the first.
  template <int SUB, int A, int FROM>
  __device__ __forceinline__ void read_after() {
    if constexpr (A == FROM - 1 || (FROM == 0 && A == 0))
      static_for<S::NR + 1 + A>([&](auto i) { read<SUB, i>(); });
    else if constexpr (A >= FROM)
      read<SUB, A + S::NR>();
  }
  template <int SUB, int A>
  __device__ __forceinline__ void group(f32x4 (&acc)[MREP][S::NR]) {
#pragma unroll
    for (int u = 0; u < S::NR; ++u)
      acc[A][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[SUB][u], q[A], acc[A][u], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  }

  // Start the first tile's first ST stages.
  __device__ __forceinline__ void begin(uint8_t* smem, const PS& P, const QS& Q) {
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_address(smem));
    const int w = wave_id(), wm = w % S::WM, wn = w / S::WM;
    PS::template read_bases<16>(pat, lds, wn * S::kWaveN);
    QS::template read_bases<kStep>(qat, lds + PS::kBytes, wm * 16);
    dest = opaque_scalar(lds + w * 1024);
    cur = 0;
#pragma unroll
    for (int st = 0; st < ST; ++st) {
      const i32x4 pr = P.template stage_resource<false>(st), qr = Q.template stage_resource<false>(st);
      static_for<kLoads>([&](auto j) { load<j, false>(P, Q, st, st, pr, qr); });
    }
  }
  // Wait for the first of them and read its first half.
  __device__ __forceinline__ void first_half() {
    stage_ready<(ST - 1) * kLoads>();
    move_by(0);
    static_for<S::NR + MREP>([&](auto i) { read<0, i>(); });
  }

  // P, Q: the sides the loads of stage `it` go by.
  template <bool WHOLE>
  __device__ __forceinline__ void step(f32x4 (&acc)[MREP][S::NR], const PS& P, const QS& Q, int it) {
    static_for<MREP>([&](auto a) {
      group<0, a>(acc);
      read_after<1, a, 0>();
      __builtin_amdgcn_sched_barrier(0);
    });
    const int nxt = cur == ST - 1 ? 0 : cur + 1;
    i32x4 pr, qr;
    static_for<MREP>([&](auto a) {
      group<1, a>(acc);
      if constexpr (a == kHead - 1) {
        move_by((nxt - cur) * kStage);
        pr = P.template stage_resource<WHOLE>(it);
        qr = Q.template stage_resource<WHOLE>(it);
        stage_ready<(ST - 2) * kLoads>();
      }
      read_after<0, a, kHead>();
      static_for<kLoads>([&](auto j) {
        constexpr int at = kHead - 1 + j * (MREP - kHead + 1) / kLoads;
        if constexpr (a == at) load<j, WHOLE>(P, Q, cur, it, pr, qr);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    cur = nxt;
  }

  // acc = the product over P's and Q's n >= ST stages; the stages that follow are those of PN and QN.
  __device__ __forceinline__ void run(f32x4 (&acc)[MREP][S::NR], const PS& P, const QS& Q, int n,
                                      const PS& PN, const QS& QN) {
#pragma unroll
    for (int a = 0; a < MREP; ++a)
#pragma unroll
      for (int b = 0; b < S::NR; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int fast = min(P.whole, Q.whole);
    int it = ST;
    for (; it < fast; ++it) step<true>(acc, P, Q, it);
    for (; it < n; ++it) step<false>(acc, P, Q, it);
    for (; it < n + ST; ++it) step<false>(acc, PN, QN, it - n);
  }
};

// One tile alone.
template <typename S, int MREP, typename PS, typename QS>
__device__ __forceinline__ void product(f32x4 (&acc)[MREP][S::NR], uint8_t* smem, const PS& P,
                                        const QS& Q, int64_t K) {
  Pipe<S, MREP, PS, QS> pipe;
  pipe.begin(smem, P, Q);
  pipe.first_half();
#pragma unroll
  for (int a = 0; a < MREP; ++a)
#pragma unroll
    for (int b = 0; b < S::NR; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int ST = Pipe<S, MREP, PS, QS>::ST;
  const int n = int((K + kBK - 1) / kBK), fast = min(P.whole, Q.whole);
  int it = ST;
  for (; it < fast; ++it) pipe.template step<true>(acc, P, Q, it);
  for (; it < n + ST; ++it) pipe.template step<false>(acc, P, Q, it);
  // Loads still under way write zeros to LDS, and other waves may still read it: both end before it
  // is used again.
  stage_ready<0>();
}

__device__ __forceinline__ u32x4 pack8(f32x4 a, f32x4 b) {
  return u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]),
               pack_bf16x2(b[2], b[3])};
}
__device__ __forceinline__ void store8(uint16_t* p, f32x4 a, f32x4 b) {
  *reinterpret_cast<u32x4*>(p) = pack8(a, b);
}
__device__ __forceinline__ void load8(const uint16_t* p, f32x4& a, f32x4& b) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(p);
  a = f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
  b = f32x4{bf16_lo(v[2]), bf16_hi(v[2]), bf16_lo(v[3]), bf16_hi(v[3])};
}

__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  const u32x2 v = *reinterpret_cast<const u32x2*>(p);
  return f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
}

template <int ACT>
__device__ __forceinline__ f32x4 act4(f32x4 v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = act_value<ACT>(v[i]);
  return v;
}

// f(m, n, v) with the sums of 8 consecutive positions from tile position n of tile row m on in v[0],
// v[1]; GATED: n is the column among the tile's gate columns, v[2], v[3] the same columns' up.  Rows
// from `rows` on are left out.
//
// The sums go through LDS, FRAGS (or up to 4) row fragments of a wave at a time,
// each wave through a part of its own: what follows is then one loop over rows, whole rows of a wave
// (256 bytes of bf16) leave together, and an activation's code is there once and not for each of 256
// registers.  It costs 2 us of a 256 x 256 tile's 60 to 200 us.  Chunk c (16 bytes) of row r sits in
// slot c ^ (r & 15), so that the 16 rows that one write serves differ in their banks.
template <typename S, bool GATED, int FRAGS = 0, int MREP, typename F>
__device__ __forceinline__ void each_row(const f32x4 (&acc)[MREP][S::NR], uint8_t* smem, int rows,
                                         F f) {
  constexpr int kFrags = FRAGS ? FRAGS : MREP <= 4 ? MREP : MREP % 3 == 0 ? 3 : 4;
  static_assert(MREP % kFrags == 0, "");
  constexpr int kRowBytes = S::kWaveN * 4, kPart = kFrags * 16 * kRowBytes;
  constexpr int kLanes = S::kWaveN / (GATED ? 16 : 8);  // lanes of one row
  const int w = wave_id(), wm = w % S::WM, wn = w / S::WM, l = lane_id();
  uint8_t* part = smem + w * kPart;
  auto chunk = [&](int r, int c) {
    return reinterpret_cast<f32x4*>(part + r * kRowBytes + ((c ^ (r & 15)) * 16));
  };
  static_for<MREP / kFrags>([&](auto pass) {
    static_for<kFrags>([&](auto a) {
      static_for<S::NR>([&](auto u) {
        *chunk(a * 16 + l % 16, u * 4 + l / 16) = acc[pass * kFrags + a][u];
      });
    });
    // a few rows a lane at a time, so that their reads are under way together
    constexpr int kRows = kWave / kLanes, kSteps = kFrags * 16 / kRows;
    constexpr int kBatch = kSteps % 4 == 0 ? 4 : kSteps % 3 == 0 ? 3 : kSteps;
    static_assert(kSteps % kBatch == 0 && kBatch <= 4, "rows of a pass in whole batches");
    const int j = l % kLanes;
#pragma unroll 1
    for (int r0 = l / kLanes; r0 < kFrags * 16; r0 += kRows * kBatch) {
      f32x4 v[kBatch][GATED ? 4 : 2];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = r0 + b * kRows;
        if constexpr (GATED) {
          const int c = (j / 4) * 16 + (j % 4) * 2;  // 32 gate columns, then the same 32 up columns
          v[b][0] = *chunk(r, c);
          v[b][1] = *chunk(r, c + 1);
          v[b][2] = *chunk(r, c + 8);
          v[b][3] = *chunk(r, c + 9);
        } else {
          v[b][0] = *chunk(r, j * 2);
          v[b][1] = *chunk(r, j * 2 + 1);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = r0 + b * kRows;
        const int m = ((pass * kFrags + r / 16) * S::WM + wm) * 16 + r % 16;
        if (m < rows) f(m, wn * (GATED ? S::kWaveN / 2 : S::kWaveN) + j * 8, v[b]);
      }
    }
  });
}

// f<MREP>() with the fewest row fragments out of a few choices that cover `rows`.
template <typename S, typename F>
__device__ __forceinline__ void by_height(int rows, F f) {
  const int need = (rows + 16 * S::WM - 1) / (16 * S::WM);
  if constexpr (S::MR >= 9)
    if (need > 8) return f(std::integral_constant<int, 9>{});
  if constexpr (S::MR >= 8)
    if (need > 6) return f(std::integral_constant<int, 8>{});
  if constexpr (S::MR >= 6)
    if (need > 4) return f(std::integral_constant<int, 6>{});
  if constexpr (S::MR >= 4)
    if (need > 2) return f(std::integral_constant<int, 4>{});
  if constexpr (S::MR >= 2)
    if (need > 1) return f(std::integral_constant<int, 2>{});
  f(std::integral_constant<int, 1>{});
}

// h = act(x Wg^T) * (x Wu^T): each wave's 64 positions are 32 gate columns and the same 32 up
// columns, so that one lane has both factors.
template <typename S>
__global__ __launch_bounds__(S::kThreads, 2) void gated_kernel(
    const uint16_t* x, const int32_t* off, const uint16_t* w, int64_t rows, int E, int H, int I,
    int act, uint16_t* h, uint16_t* gu) {
  __shared__ __align__(1024) uint8_t smem[S::kLds];
  constexpr int kCols = S::BN / 2;
  const int ncol = (I + kCols - 1) / kCols;
  for (uint32_t id = blockIdx.x;; id += gridDim.x) {
    const Tile t = find_tile<S::FULL, S::BM, S::kThreads>(off, E, rows, ncol, id);
    if (t.e < 0) return;
    const int n0 = t.nt * kCols;
    const uint16_t* we = w + (int64_t(t.e) * 2 * I + n0) * H;
    Side<true, S::BN, S::W, true, S::kOnce> P;
    P.init_kc(we, we + int64_t(I) * H, H, H, I - n0);
    const uint16_t* xe = x + t.row0 * H;
    by_height<S>(t.rows, [&](auto mrep) {
      constexpr int M = decltype(mrep)::value;
      Side<true, S::template kRows<M>, S::W> Q;
      Q.init_kc(xe, xe, H, H, t.rows);
      f32x4 acc[M][S::NR];
      product<S, M>(acc, smem, P, Q, H);
      with_act(act, [&](auto a) {
        if constexpr (a != MOE_ACT_NONE)
          each_row<S, true>(acc, smem, t.rows, [&](int m, int c, const f32x4(&v)[4]) {
            const int n = n0 + c;
            if (n >= I) return;
            const int64_t row = t.row0 + m;
            store8(h + row * I + n, act4<a>(v[0]) * v[2], act4<a>(v[1]) * v[3]);
            if (gu != nullptr) {
              store8(gu + row * 2 * I + n, v[0], v[1]);
              store8(gu + row * 2 * I + I + n, v[2], v[3]);
            }
          });
      });
    });
  }
}

// y = act(x W^T + bias) + residual, pre = act's argument.
template <typename S>
__global__ __launch_bounds__(S::kThreads, 2) void matmul_kernel(
    const uint16_t* x, const int32_t* off, const uint16_t* w, const uint16_t* bias,
    const uint16_t* res, int64_t rows, int E, int K, int N, int act, uint16_t* y, uint16_t* pre) {
  __shared__ __align__(1024) uint8_t smem[S::kLds];
  const int ncol = (N + S::BN - 1) / S::BN;
  for (uint32_t id = blockIdx.x;; id += gridDim.x) {
    const Tile t = find_tile<S::FULL, S::BM, S::kThreads>(off, E, rows, ncol, id);
    if (t.e < 0) return;
    const int n0 = t.nt * S::BN;
    const uint16_t* we = w + (int64_t(t.e) * N + n0) * K;
    const uint16_t* xe = x + t.row0 * K;
    Side<true, S::BN, S::W, false, S::kOnce> P;
    P.init_kc(we, we, K, K, N - n0);
    by_height<S>(t.rows, [&](auto mrep) {
      constexpr int M = decltype(mrep)::value;
      Side<true, S::template kRows<M>, S::W> Q;
      Q.init_kc(xe, xe, K, K, t.rows);
      f32x4 acc[M][S::NR];
      product<S, M>(acc, smem, P, Q, K);
      with_act(act, [&](auto a) {
        each_row<S, false>(acc, smem, t.rows, [&](int m, int c, const f32x4(&v)[2]) {
          const int n = n0 + c;
          if (n >= N) return;
          const int64_t at = (t.row0 + m) * N + n;
          f32x4 v0 = v[0], v1 = v[1], r0, r1;
          if (bias != nullptr) {
            load8(bias + int64_t(t.e) * N + n, r0, r1);
            v0 += r0;
            v1 += r1;
          }
          if (pre != nullptr) store8(pre + at, v0, v1);
          v0 = act4<a>(v0);
          v1 = act4<a>(v1);
          if (res != nullptr) {
            load8(res + at, r0, r1);
            v0 += r0;
            v1 += r1;
          }
          store8(y + at, v0, v1);
        });
      });
    });
  }
}

// The forward products where few rows meet few outputs: 32 rows by 32 positions (gated: 16 gate
// columns and the same 16 up columns) a block, the inner axis split over its 8 waves.  Each wave takes
// every 8th piece of 32 k straight from memory into the matrix instruction's registers, kAhead pieces
// at a time; the 8 partial sums meet in LDS and are added in the waves' order.  With few blocks on the
// chip the time is that of one block, and what bounds it is how often a wave waits for memory: 8 waves
// of 4 pieces wait once per 1024 k, where the 128x128 tiles do per 64 (16 experts of 128 x 2312, 32
// rows: 13.1 against 7.9 us, 4 us of either the launch's).
constexpr int kThinRows = 32, kThinCols = 32, kThinWaves = 8;

template <bool GATED>
__global__ __launch_bounds__(kThinWaves * kWave) void thin_kernel(
    const uint16_t* x, const int32_t* off, const uint16_t* w, const uint16_t* bias,
    const uint16_t* res, int64_t rows, int E, int K, int N, int act, uint16_t* y, uint16_t* pre) {
  constexpr int kAhead = 4, kCols = GATED ? kThinCols / 2 : kThinCols;
  __shared__ f32x4 part[kThinWaves][4][kWave];
  const int ncol = (N + kCols - 1) / kCols;
  const int wv = wave_id(), l = lane_id(), i = l % 16, q = l / 16;
  for (uint32_t id = blockIdx.x;; id += gridDim.x) {
    const Tile t = find_tile<kThinRows, kThinRows, kThinWaves * kWave>(off, E, rows, ncol, id);
    if (t.e < 0) return;
    const int n0 = t.nt * kCols;
    // Rows and columns outside the tile repeat its last one; their sums are not stored.
    const uint16_t *wp[2], *xp[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int n = n0 + (GATED ? 0 : f * 16) + i, m = f * 16 + i;
      wp[f] = w + (int64_t(t.e) * (GATED ? 2 : 1) * N + (GATED ? f * int64_t(N) : 0) +
                   (n < N ? n : N - 1)) * K + q * 8;
      xp[f] = x + (t.row0 + (m < t.rows ? m : t.rows - 1)) * K + q * 8;
    }
    f32x4 acc[2][2] = {};
    for (int k0 = wv * 32; k0 < K; k0 += kThinWaves * 32 * kAhead) {
      u32x4 a[kAhead][2], b[kAhead][2];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * kThinWaves * 32;
        const bool in = k + q * 8 < K;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          a[u][f] = b[u][f] = u32x4{0u, 0u, 0u, 0u};
          if (in) {
            a[u][f] = *reinterpret_cast<const u32x4*>(wp[f] + k);
            b[u][f] = *reinterpret_cast<const u32x4*>(xp[f] + k);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            acc[f][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, a[u][f]), __builtin_bit_cast(bf16x8, b[u][m]),
                acc[f][m], 0, 0, 0);
    }
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int m = 0; m < 2; ++m) part[wv][f * 2 + m][l] = acc[f][m];
    __syncthreads();
    // waves 0 and 1 finish the two row fragments (gated: both factors), or waves 0 to 3 a fragment each
    const int m = wv % 2 * 16 + i;
    if (wv < (GATED ? 2 : 4) && m < t.rows) {
      auto sum = [&](int f) {
        f32x4 v = part[0][f * 2 + wv % 2][l];
#pragma unroll
        for (int s = 1; s < kThinWaves; ++s) v += part[s][f * 2 + wv % 2][l];
        return v;
      };
      const int64_t row = t.row0 + m;
      if constexpr (GATED) {
        const int n = n0 + q * 4;
        const f32x4 g = sum(0), u = sum(1);
        if (n < N) {
          with_act(act, [&](auto c) { store4(y + row * N + n, act4<c>(g) * u); });
          if (pre != nullptr) {
            store4(pre + row * 2 * N + n, g);
            store4(pre + row * 2 * N + N + n, u);
          }
        }
      } else {
        const int n = n0 + wv / 2 * 16 + q * 4;
        f32x4 v = sum(wv / 2);
        if (n < N) {
          const int64_t at = row * N + n;
          if (bias != nullptr) v += load4(bias + int64_t(t.e) * N + n);
          if (pre != nullptr) store4(pre + at, v);
          with_act(act, [&](auto c) { v = act4<c>(v); });
          if (res != nullptr) v += load4(res + at);
          store4(y + at, v);
        }
      }
    }
    __syncthreads();  // part may be written again
  }
}

// Tile number `id` of dx = d W: the weights [N, K] are contiguous along the output's own index.  False
// behind the last tile.
template <typename S>
__device__ __forceinline__ bool data_grad_tile(uint32_t id, uint8_t* smem, const uint16_t* d,
                                               const int32_t* off, const uint16_t* w, int64_t rows,
                                               int E, int N, int K, uint16_t* dx) {
  const Tile t = find_tile<S::FULL, S::BM, S::kThreads>(off, E, rows, (K + S::BN - 1) / S::BN, id);
  if (t.e < 0) return false;
  const int n0 = t.nt * S::BN;
  const uint16_t* we = w + int64_t(t.e) * N * K + n0;
  const uint16_t* de = d + t.row0 * N;
  Side<false, S::BN, S::W, false, S::kOnce> P;
  P.init_mc(we, K, N, n0);
  by_height<S>(t.rows, [&](auto mrep) {
    constexpr int M = decltype(mrep)::value;
    Side<true, S::template kRows<M>, S::W> Q;
    Q.init_kc(de, de, N, N, t.rows);
    f32x4 acc[M][S::NR];
    product<S, M>(acc, smem, P, Q, N);
    each_row<S, false>(acc, smem, t.rows, [&](int m, int c, const f32x4(&v)[2]) {
      if (n0 + c < K) store8(dx + (t.row0 + m) * K + n0 + c, v[0], v[1]);
    });
  });
  return true;
}

template <typename S>
__global__ __launch_bounds__(S::kThreads, 2) void data_grad_kernel(
    const uint16_t* d, const int32_t* off, const uint16_t* w, int64_t rows, int E, int N, int K,
    uint16_t* dx) {
  __shared__ __align__(1024) uint8_t smem[S::kLds];
  for (uint32_t id = blockIdx.x; data_grad_tile<S>(id, smem, d, off, w, rows, E, N, K, dx);
       id += gridDim.x) {
  }
}

// dW[e] = d^T x over the expert's rows: both sides are contiguous along the
// output's indexes.  An expert without rows gets zeros.
//
// With some hundred rows an expert a tile is over after a few stages, and its start (2 us until the
// first loads arrive) and its end (5 us of stores) cost as much as its product.  So one block a CU
// goes through its tiles as one sequence of stages: the next tile's first stages arrive while the
// current one's last are computed, and the sums leave through LDS of their own while they do.  A
// tile is at least ST stages long for that, the added ones all zeros.
template <typename S, bool F32>
__global__ __launch_bounds__(S::kThreads, 2) void weight_grad_kernel(
    const uint16_t* d, const uint16_t* x, const int32_t* off, int64_t rows, int E, int N, int K,
    void* dw) {
  typedef Side<false, S::BN, S::W> PS;
  typedef Side<false, S::BM, S::W> QS;
  typedef Pipe<S, S::MR, PS, QS> Pipeline;
  __shared__ __align__(1024) uint8_t smem[Pipeline::ST * Pipeline::kStage];
  __shared__ __align__(1024) uint8_t sums[S::W * 16 * S::kWaveN * 4];
  const uint32_t nn = (N + S::BM - 1) / S::BM, nk = (K + S::BN - 1) / S::BN;
  const uint32_t total = E * nn * nk;
  struct Place {
    uint32_t id;
    int e, m0, n0, n;  // n stages; 0 behind the last tile
  };
  auto put = [&](const Place& t, int m, int c, const f32x4(&v)[2]) {
    if (t.n0 + c >= K) return;
    const int64_t at = (int64_t(t.e) * N + t.m0 + m) * K + t.n0 + c;
    if (F32) {
      f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(dw) + at);
      o[0] = v[0];
      o[1] = v[1];
    } else {
      store8(static_cast<uint16_t*>(dw) + at, v[0], v[1]);
    }
  };
  // The first tile from number `id` on that has rows, and its sides; tiles without are written on the
  // way.
  auto find = [&](uint32_t id, Place& t, PS& P, QS& Q) {
    t = Place{};
    int64_t lo = 0, cnt = 0;
    for (; id < total; id += gridDim.x) {
      const uint32_t seq = xcd_order(id, total);
      t.e = int(seq / (nn * nk));
      int mt, ct;
      grid_order(seq - uint32_t(t.e) * nn * nk, nn, nk, mt, ct);
      t.m0 = mt * S::BM;
      t.n0 = ct * S::BN;
      expert_rows_scalar(off, t.e, rows, lo, cnt);
      if (cnt > 0) break;
      const f32x4 zero[2] = {};
      for (int i = threadIdx.x; i < S::BM * (S::BN / 8); i += S::kThreads) {
        const int m = i / (S::BN / 8);
        if (t.m0 + m < N) put(t, m, i % (S::BN / 8) * 8, zero);
      }
    }
    t.id = id;
    if (cnt > 0) {
      const int n = int((cnt + kBK - 1) / kBK);
      t.n = n < Pipeline::ST ? Pipeline::ST : n;
    }
    P.init_mc(x + lo * K + t.n0, K, cnt, t.n0);
    Q.init_mc(d + lo * N + t.m0, N, cnt, t.m0);
  };
  Place t, next;
  PS P, PN;
  QS Q, QN;
  find(blockIdx.x, t, P, Q);
  if (t.n == 0) return;
  Pipeline pipe;
  pipe.begin(smem, P, Q);
  pipe.first_half();
  f32x4 acc[S::MR][S::NR];
  do {
    find(t.id + gridDim.x, next, PN, QN);
    pipe.run(acc, P, Q, t.n, PN, QN);
    each_row<S, false, 1>(acc, sums, N - t.m0, [&](int m, int c, const f32x4(&v)[2]) {
      put(t, m, c, v);
    });
    t = next;
    P = PN;
    Q = QN;
  } while (t.n > 0);
  stage_ready<0>();  // the loads behind the last tile
}

// One tile of the same, for a block of its own.
template <typename S, bool F32>
__device__ __forceinline__ void weight_grad_tile(uint32_t id, uint8_t* smem, const uint16_t* d,
                                                 const uint16_t* x, const int32_t* off,
                                                 int64_t rows, int E, int N, int K, void* dw) {
  const uint32_t nn = (N + S::BM - 1) / S::BM, nk = (K + S::BN - 1) / S::BN;
  const uint32_t seq = xcd_order(id, E * nn * nk);
  const int e = int(seq / (nn * nk));
  int mt, ct;
  grid_order(seq - uint32_t(e) * nn * nk, nn, nk, mt, ct);
  const int m0 = mt * S::BM, n0 = ct * S::BN;
  int64_t lo, cnt;
  expert_rows_scalar(off, e, rows, lo, cnt);
  f32x4 acc[S::MR][S::NR] = {};
  if (cnt > 0) {
    Side<false, S::BN, S::W> P;
    Side<false, S::BM, S::W> Q;
    P.init_mc(x + lo * K + n0, K, cnt, n0);
    Q.init_mc(d + lo * N + m0, N, cnt, m0);
    product<S, S::MR>(acc, smem, P, Q, cnt);
  }
  each_row<S, false>(acc, smem, N - m0, [&](int m, int c, const f32x4(&v)[2]) {
    if (n0 + c >= K) return;
    const int64_t at = (int64_t(e) * N + m0 + m) * K + n0 + c;
    if (F32) {
      f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(dw) + at);
      o[0] = v[0];
      o[1] = v[1];
    } else {
      store8(static_cast<uint16_t*>(dw) + at, v[0], v[1]);
    }
  });
}

// Both gradients of a small product in one launch, a block a tile: the first `data_blocks` blocks
// those of dx, the others those of dW.  Neither fills the chip, and each is over after one tile's time
// (matmul_backward of 300 rows, 16 experts of 1288 x 520, with its elementwise part: 34.6 us with
// a launch each, 23.9 with one).
template <typename S, bool F32>
__global__ __launch_bounds__(S::kThreads, 2) void both_grads_kernel(
    const uint16_t* d, const uint16_t* x, const int32_t* off, const uint16_t* w, int64_t rows, int E,
    int N, int K, uint32_t data_blocks, uint16_t* dx, void* dw) {
  __shared__ __align__(1024) uint8_t smem[S::kLds];
  if (blockIdx.x < data_blocks)
    data_grad_tile<S>(blockIdx.x, smem, d, off, w, rows, E, N, K, dx);
  else
    weight_grad_tile<S, F32>(blockIdx.x - data_blocks, smem, d, x, off, rows, E, N, K, dw);
}

template <typename S, bool F32>
__global__ __launch_bounds__(S::kThreads, 2) void weight_grad_alone_kernel(
    const uint16_t* d, const uint16_t* x, const int32_t* off, int64_t rows, int E, int N, int K,
    void* dw) {
  __shared__ __align__(1024) uint8_t smem[S::kLds];
  weight_grad_tile<S, F32>(blockIdx.x, smem, d, x, off, rows, E, N, K, dw);
}

// ---------------------------------------------------------------------------
// elementwise gradients
// ---------------------------------------------------------------------------

// [dg du] from dh and the kept factors, 8 columns per thread.
template <int ACT>
__global__ __launch_bounds__(256) void gated_grad_kernel(const uint16_t* dh, const uint16_t* gu,
                                                         const int32_t* off, int64_t rows, int E,
                                                         int I, uint16_t* dgu) {
  const int64_t first = off[0] < 0 ? 0 : (off[0] > rows ? rows : off[0]);
  const int64_t last = off[E] < 0 ? 0 : (off[E] > rows ? rows : off[E]);
  const int C = I / 8;
  const int64_t total = (last - first) * C;
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t row = first + i / C;
    const int64_t c = i % C * 8;
    const u32x4 vh = *reinterpret_cast<const u32x4*>(dh + row * I + c);
    const u32x4 vg = *reinterpret_cast<const u32x4*>(gu + row * 2 * I + c);
    const u32x4 vu = *reinterpret_cast<const u32x4*>(gu + row * 2 * I + I + c);
    u32x4 og, ou;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float h0 = bf16_lo(vh[q]), h1 = bf16_hi(vh[q]);
      const float g0 = bf16_lo(vg[q]), g1 = bf16_hi(vg[q]);
      og[q] = pack_bf16x2(h0 * bf16_lo(vu[q]) * act_slope<ACT>(g0),
                          h1 * bf16_hi(vu[q]) * act_slope<ACT>(g1));
      ou[q] = pack_bf16x2(h0 * act_value<ACT>(g0), h1 * act_value<ACT>(g1));
    }
    *reinterpret_cast<u32x4*>(dgu + row * 2 * I + c) = og;
    *reinterpret_cast<u32x4*>(dgu + row * 2 * I + I + c) = ou;
  }
}

// dpre = dy * act'(pre), 8 columns per thread.
template <int ACT>
__global__ __launch_bounds__(256) void pre_kernel(const uint16_t* dy, const uint16_t* pre,
                                                  const int32_t* off, int64_t rows, int E, int N,
                                                  uint16_t* dpre) {
  const int64_t first = off[0] < 0 ? 0 : (off[0] > rows ? rows : off[0]);
  const int64_t last = off[E] < 0 ? 0 : (off[E] > rows ? rows : off[E]);
  const int64_t end = last * N;
  for (int64_t at = first * N + (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) * 8; at < end;
       at += int64_t(gridDim.x) * blockDim.x * 8) {
    f32x4 y0, y1, p0, p1;
    load8(dy + at, y0, y1);
    load8(pre + at, p0, p1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y0[i] *= act_slope<ACT>(p0[i]);
      y1[i] *= act_slope<ACT>(p1[i]);
    }
    store8(dpre + at, y0, y1);
  }
}

// The same with dbias[e], dpre's sum over the expert's rows, in a fixed order: a block owns COLS columns
// of one expert, COLS / 8 threads a row, each thread adding every (8 THREADS / COLS)th row, then the
// lanes of a wave by a butterfly and the waves in their order.  What bounds it with few experts is the
// one CU's work on a strip, so strips are then narrower and blocks larger (see the launch).
template <int ACT, int THREADS, int COLS>
__global__ __launch_bounds__(THREADS) void pre_grad_kernel(const uint16_t* dy, const uint16_t* pre,
                                                           const int32_t* off, int64_t rows, int E,
                                                           int N, uint16_t* dpre, float* dbias) {
  constexpr int kLanes = COLS / 8, kStep = THREADS / kLanes, kAhead = THREADS > 256 ? 4 : 1;
  __shared__ float part[THREADS / kWave][COLS];
  const int64_t strips = (N + COLS - 1) / COLS;
  for (int64_t u = blockIdx.x; u < E * strips; u += gridDim.x) {
    const int e = int(u / strips), strip = int(u % strips) * COLS;
    const int c = strip + int(threadIdx.x) % kLanes * 8;
    int64_t lo, cnt;
    expert_rows(off, e, rows, lo, cnt);
    f32x4 s0 = {}, s1 = {};
    if (c < N) {
      for (int64_t r = threadIdx.x / kLanes; r < cnt; r += kStep * kAhead) {
        f32x4 y0[kAhead], y1[kAhead], p0[kAhead] = {}, p1[kAhead] = {};
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          y0[i] = y1[i] = f32x4{};
          if (r + i * kStep < cnt) {
            const int64_t at = (lo + r + i * kStep) * N + c;
            load8(dy + at, y0[i], y1[i]);
            if (ACT != MOE_ACT_NONE) load8(pre + at, p0[i], p1[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (r + i * kStep >= cnt) continue;
          if (ACT != MOE_ACT_NONE) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y0[i][j] *= act_slope<ACT>(p0[i][j]);
              y1[i][j] *= act_slope<ACT>(p1[i][j]);
            }
            store8(dpre + (lo + r + i * kStep) * N + c, y0[i], y1[i]);
          }
          s0 += y0[i];
          s1 += y1[i];
        }
      }
    }
#pragma unroll
    for (int m = kLanes; m < kWave; m <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s0[j] += __shfl_xor(s0[j], m);
        s1[j] += __shfl_xor(s1[j], m);
      }
    __syncthreads();  // part of the strip before has been read
    if (lane_id() < kLanes) {
      f32x4* o = reinterpret_cast<f32x4*>(&part[threadIdx.x / kWave][lane_id() * 8]);
      o[0] = s0;
      o[1] = s1;
    }
    __syncthreads();
    if (threadIdx.x < COLS && strip + int(threadIdx.x) < N) {
      float s = 0.f;
      for (int w = 0; w < THREADS / kWave; ++w) s += part[w][threadIdx.x];
      dbias[int64_t(e) * N + strip + threadIdx.x] = s;
    }
  }
}

// combine's gradient, one wave per (token, j): dy[row] = bf16(w dout[t]) and
// dw = sum over the columns of dout[t] * y[row], each lane adding its own
// columns in ascending order and the lanes' sums meeting in a fixed butterfly.
__global__ __launch_bounds__(256) void combine_grad_kernel(
    const u32x4* __restrict__ dout, const u32x4* __restrict__ y,
    const int32_t* __restrict__ pair_row, const float* __restrict__ topk_w, int64_t T, int C,
    int k, int64_t capacity, u32x4* __restrict__ dy, float* __restrict__ dw) {
  for (int64_t p = blockIdx.x * int64_t(4) + threadIdx.x / kWave; p < T * k;
       p += gridDim.x * int64_t(4)) {
    const int64_t r = pair_row[p];
    const float w = topk_w[p];
    if (r < 0 || r >= capacity) {  // a dropped pair has no row: its weight has no effect
      if (lane_id() == 0) dw[p] = 0.f;
      continue;
    }
    const u32x4* dr = dout + (p / k) * C;
    float s0 = 0.f, s1 = 0.f;
    for (int c = lane_id(); c < C; c += kWave) {
      const u32x4 vd = dr[c];
      const u32x4 vy = __builtin_nontemporal_load(&y[r * C + c]);
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float d0 = bf16_lo(vd[q]), d1 = bf16_hi(vd[q]);
        s0 = __builtin_fmaf(d0, bf16_lo(vy[q]), s0);
        s1 = __builtin_fmaf(d1, bf16_hi(vy[q]), s1);
        o[q] = pack_bf16x2(w * d0, w * d1);
      }
      __builtin_nontemporal_store(o, &dy[r * C + c]);
    }
    float s = s0 + s1;
    for (int m = 1; m < kWave; m <<= 1) s += __shfl_xor(s, m);
    if (lane_id() == 0) dw[p] = s;
  }
}

// ---------------------------------------------------------------------------
// host side: checks and launches
// ---------------------------------------------------------------------------

template <typename Tuple, size_t... I>
void arg_ptrs(Tuple& t, void** argv, std::index_sequence<I...>) {
  ((argv[I] = static_cast<void*>(&std::get<I>(t))), ...);
}

template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), int64_t blocks, int threads, hipStream_t st, Args... args) {
  static_assert(sizeof...(KArgs) == sizeof...(Args), "kernel arity");
  const unsigned grid = unsigned(blocks < kMaxBlocks ? blocks : kMaxBlocks);
  std::tuple<KArgs...> packed(static_cast<KArgs>(args)...);
  void* argv[sizeof...(KArgs)];
  arg_ptrs(packed, argv, std::index_sequence_for<KArgs...>{});
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kern), dim3(grid),
                                       dim3(unsigned(threads)), argv, 0, st);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool bad_features(int32_t n) { return n < 8 || n > kMaxFeatures; }

// One block of 8 waves a CU: two stages of 32 KiB of weights and up to 40 KiB of rows.
template <bool ONCE>
using TallOf = Shape<256, 288, 256, 2, 4, 144 * 1024, ONCE>;
using Tall = TallOf<false>;
using Square = Shape<256, 256, 256, 2, 4, 128 * 1024>;
// 4 waves, two blocks a CU.
template <bool ONCE>
using HalfOf = Shape<128, 128, 128, 2, 2, 72 * 1024, ONCE>;
using Half = HalfOf<false>;

// The sizes every product shares; MOE_OK with rows == 0 allowed.  Tile numbers are 32-bit: what a
// call could need at most has to stay below 2^31, far beyond any buffers that fit the card.
int check_sizes(int64_t rows, int32_t E, int32_t a, int32_t b, int32_t act, bool none_ok) {
  if (rows < 0 || rows > kMaxPairs || E < 1 || E > kMaxE) return MOE_ERR_INVALID_ARG;
  if (bad_features(a) || bad_features(b)) return MOE_ERR_INVALID_ARG;
  if (act < (none_ok ? MOE_ACT_NONE : MOE_ACT_SILU) || act > MOE_ACT_RELU)
    return MOE_ERR_INVALID_ARG;
  if (a % 8 != 0 || b % 8 != 0) return MOE_ERR_ALIGNMENT;
  const int64_t ca = a / 64 + 1, cb = b / 64 + 1;  // columns of the narrowest tiles
  const int64_t tall = rows / Half::FULL + E;
  if (tall * ca > kMaxTiles || tall * cb > kMaxTiles || ca * cb > kMaxTiles / E)
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Blocks for tiles of at most `bm` rows that `rows` rows in E runs can need, `cols` to a row of
// tiles.
int64_t row_tile_blocks(int64_t rows, int32_t E, int bm, int64_t cols) {
  return (rows / bm + (rows < E ? rows : E)) * cols;
}

// Whether a product over the experts' rows takes Half tiles: under 128 rows an expert (the tall
// tiles' heights are then mostly empty, and two blocks a CU cover each other's waits), or so few tall
// tiles that half of the CUs would have none.  `per_tile`: those of the outputs' `cols` columns that a
// tall tile covers.
// Measured, rows spread at random, tall against half tiles: 64 experts of 2048 x 2048, 64 rows each,
// 142 against 127 us, 128 rows 153 against 158, 256 rows 183 against 212; 16 of 4096 x 4096, 64 rows
// 134 against 116, 128 rows 146 against 179; 8 of 520 x 1280, 512 rows 30 against 19; 8 of 2048 x 544
// (3 column tiles, 7 blocks in 8 idle), 512 rows 47 against 26.
bool half_tiles(int64_t rows, int32_t E, int64_t cols, int per_tile) {
  return rows < int64_t(E) * 128 ||
         row_tile_blocks(rows, E, Tall::FULL, (cols + per_tile - 1) / per_tile) <= kCus / 2;
}

// Whether the weights [E, N, K] go past the caches: their strips are read by one tile each (no more
// rows an expert than a tall tile holds), they are larger than the 256 MiB Infinity Cache, so that
// nothing of them is there at the next call either, and their rows are whole lines, no part of which
// is read again.  Kept against read once: 64 experts of 2048 x 4096 with 16 rows each 207 against 186
// us, 256 rows 325 against 286, 512 rows 592 against 596; rows of 1000 features (8 experts of 7168)
// 24 against 32 us.
bool read_once(int64_t rows, int32_t E, int64_t N, int64_t K) {
  return rows <= int64_t(E) * Tall::BM && E * N * K * 2 > int64_t(256) << 20 && K % 64 == 0;
}

// Whether a forward product goes to thin_kernel: its tiles, 32 rows by `per_tile` of the outputs'
// `cols` columns, number at most 3 for two CUs.  Measured, products of the other shapes against thin
// ones, rows spread at random: one expert of 512 x 1024 500 rows (256 thin tiles) 11.9 against 7.2 us,
// of 1024 x 4096 480 rows (512) 42 against 32; 4 of 2048 x 4096 4 rows (256) 20 against 13, 64 rows
// (384) 21 against 16, 128 rows (512) 23 against 32; 16 of 256 x 4096 512 rows (256) 22 against 18, all
// at one expert of 16 of 128 x 2312 (128) 21 against 9; 64 of 2048 x 1024 16 rows (1024) 12 against 16,
// all 512 at one of 16 of 1024 x 4096 (1024) 42 against 33.
bool thin_tiles(int64_t rows, int32_t E, int64_t cols, int per_tile) {
  return row_tile_blocks(rows, E, kThinRows, (cols + per_tile - 1) / per_tile) <= kCus * 3 / 2;
}

// run(shape) of the shape a product with weights [E, N, K] takes.
template <typename F>
int with_shape(int64_t rows, int32_t E, int64_t N, int64_t K, int64_t cols, int per_tile, F run) {
  const bool once = read_once(rows, E, N, K);
  if (half_tiles(rows, E, cols, per_tile))
    return once ? run(HalfOf<true>{}) : run(HalfOf<false>{});
  return once ? run(TallOf<true>{}) : run(TallOf<false>{});
}

}  // namespace

extern "C" {

int moe_expert_gated(const void* x, const int32_t* expert_offsets, const void* w_gate_up,
                     int64_t rows, int32_t E, int32_t H, int32_t I, int32_t act, void* h,
                     void* gate_up, void* stream) {
  const int st = check_sizes(rows, E, H, I, act, false);
  if (st != MOE_OK || rows == 0) return st;
  if (!x || !expert_offsets || !w_gate_up || !h) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w_gate_up, 16) || !aligned(h, 16) || !aligned(gate_up, 16) ||
      !aligned(expert_offsets, 4))
    return MOE_ERR_ALIGNMENT;
  if (thin_tiles(rows, E, I, kThinCols / 2))
    return launch(thin_kernel<true>,
                  row_tile_blocks(rows, E, kThinRows, (I + kThinCols / 2 - 1) / (kThinCols / 2)),
                  kThinWaves * kWave, static_cast<hipStream_t>(stream),
                  static_cast<const uint16_t*>(x), expert_offsets,
                  static_cast<const uint16_t*>(w_gate_up), nullptr, nullptr, rows, E, H, I, act,
                  static_cast<uint16_t*>(h), static_cast<uint16_t*>(gate_up));
  return with_shape(rows, E, 2 * I, H, I, Tall::BN / 2, [&](auto shape) {
    using S = decltype(shape);
    return launch(gated_kernel<S>,
                  row_tile_blocks(rows, E, S::FULL, (I + S::BN / 2 - 1) / (S::BN / 2)),
                  S::kThreads, static_cast<hipStream_t>(stream),
                  static_cast<const uint16_t*>(x), expert_offsets,
                  static_cast<const uint16_t*>(w_gate_up), rows, E, H, I, act,
                  static_cast<uint16_t*>(h), static_cast<uint16_t*>(gate_up));
  });
}

int moe_expert_matmul(const void* x, const int32_t* expert_offsets, const void* w,
                      const void* bias, const void* residual, int64_t rows, int32_t E, int32_t K,
                      int32_t N, int32_t act, void* y, void* pre, void* stream) {
  const int st = check_sizes(rows, E, K, N, act, true);
  if (st != MOE_OK || rows == 0) return st;
  if (!x || !expert_offsets || !w || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(bias, 16) ||
      !aligned(residual, 16) || !aligned(pre, 16) || !aligned(expert_offsets, 4))
    return MOE_ERR_ALIGNMENT;
  if (thin_tiles(rows, E, N, kThinCols))
    return launch(thin_kernel<false>,
                  row_tile_blocks(rows, E, kThinRows, (N + kThinCols - 1) / kThinCols),
                  kThinWaves * kWave, static_cast<hipStream_t>(stream),
                  static_cast<const uint16_t*>(x), expert_offsets,
                  static_cast<const uint16_t*>(w), static_cast<const uint16_t*>(bias),
                  static_cast<const uint16_t*>(residual), rows, E, K, N, act,
                  static_cast<uint16_t*>(y), static_cast<uint16_t*>(pre));
  return with_shape(rows, E, N, K, N, Tall::BN, [&](auto shape) {
    using S = decltype(shape);
    return launch(matmul_kernel<S>, row_tile_blocks(rows, E, S::FULL, (N + S::BN - 1) / S::BN),
                  S::kThreads, static_cast<hipStream_t>(stream), static_cast<const uint16_t*>(x),
                  expert_offsets, static_cast<const uint16_t*>(w),
                  static_cast<const uint16_t*>(bias), static_cast<const uint16_t*>(residual), rows,
                  E, K, N, act, static_cast<uint16_t*>(y), static_cast<uint16_t*>(pre));
  });
}

// dx = d W and dW = d^T x, either of which may be left out (NULL).
static int product_grads(const void* d, const void* x, const int32_t* off, const void* w,
                         int64_t rows, int E, int N, int K, void* dx, void* dw, int dw_f32,
                         hipStream_t s) {
  const uint16_t* dv = static_cast<const uint16_t*>(d);
  const uint16_t* xv = static_cast<const uint16_t*>(x);
  const uint16_t* wv = static_cast<const uint16_t*>(w);
  uint16_t* dxv = static_cast<uint16_t*>(dx);
  if (rows == 0) dx = nullptr;
  auto tiles = [&](int side) {
    return int64_t(E) * ((N + side - 1) / side) * ((K + side - 1) / side);
  };
  // So few square tiles that they fill the CUs once at best go in halves, a block each: 16 experts of
  // 1288 x 520 (288 square tiles) take 12.0 us in halves, 15.8 as square ones with a block each; 64 of
  // 2048 x 2048 take 123 us in one sequence of square tiles a CU, 152 with a block each, 173 in halves
  // (16 rows an expert), and 235, 260 and 310 us (256 rows).
  const bool halves = tiles(Square::BM) <= kCus + kCus / 4;
  if (dx && dw && halves && half_tiles(rows, E, K, Tall::BN)) {
    const int64_t nd = row_tile_blocks(rows, E, Half::FULL, (K + Half::BN - 1) / Half::BN);
    const int64_t n = nd + tiles(Half::BM);
    if (n <= kMaxBlocks)
      return launch(dw_f32 ? both_grads_kernel<Half, true> : both_grads_kernel<Half, false>, n,
                    Half::kThreads, s, dv, xv, off, wv, rows, E, N, K, uint32_t(nd), dxv, dw);
  }
  int st = MOE_OK;
  if (dx)
    st = with_shape(rows, E, N, K, K, Tall::BN, [&](auto shape) {
      using S = decltype(shape);
      return launch(data_grad_kernel<S>, row_tile_blocks(rows, E, S::FULL, (K + S::BN - 1) / S::BN),
                    S::kThreads, s, dv, off, wv, rows, E, N, K, dxv);
    });
  if (st != MOE_OK || !dw) return st;
  if (halves)
    return launch(
        dw_f32 ? weight_grad_alone_kernel<Half, true> : weight_grad_alone_kernel<Half, false>,
        tiles(Half::BM), Half::kThreads, s, dv, xv, off, rows, E, N, K, dw);
  const int64_t n = tiles(Square::BM);
  return launch(dw_f32 ? weight_grad_kernel<Square, true> : weight_grad_kernel<Square, false>,
                n < kCus ? n : kCus, Square::kThreads, s, dv, xv, off, rows, E, N, K, dw);
}

int moe_expert_gated_backward(const void* dh, const void* gate_up, const void* x,
                              const int32_t* expert_offsets, const void* w_gate_up, int64_t rows,
                              int32_t E, int32_t H, int32_t I, int32_t act, void* dgate_up,
                              void* dx, void* dw, int32_t dw_f32, void* stream) {
  int st = check_sizes(rows, E, H, I, act, false);
  if (st != MOE_OK) return st;
  if (!expert_offsets || (dw_f32 != 0 && dw_f32 != 1)) return MOE_ERR_INVALID_ARG;
  if (rows > 0) {
    if (!dh || !gate_up || !dgate_up || (dx && !w_gate_up) || (dw && !x))
      return MOE_ERR_INVALID_ARG;
  }
  if (!aligned(dh, 16) || !aligned(gate_up, 16) || !aligned(x, 16) || !aligned(w_gate_up, 16) ||
      !aligned(dgate_up, 16) || !aligned(dx, 16) || !aligned(dw, 16) ||
      !aligned(expert_offsets, 4))
    return MOE_ERR_ALIGNMENT;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows > 0) {
    auto kern = act == MOE_ACT_SILU   ? gated_grad_kernel<MOE_ACT_SILU>
                : act == MOE_ACT_GELU ? gated_grad_kernel<MOE_ACT_GELU>
                                      : gated_grad_kernel<MOE_ACT_RELU>;
    st = launch(kern, (rows * (I / 8) + 255) / 256, 256, s,
                static_cast<const uint16_t*>(dh), static_cast<const uint16_t*>(gate_up),
                expert_offsets, rows, E, I, static_cast<uint16_t*>(dgate_up));
  }
  if (st != MOE_OK) return st;
  return product_grads(dgate_up, x, expert_offsets, w_gate_up, rows, E, 2 * I, H, dx, dw, dw_f32, s);
}

int moe_expert_matmul_backward(const void* dy, const void* pre, const void* x,
                               const int32_t* expert_offsets, const void* w, int64_t rows,
                               int32_t E, int32_t K, int32_t N, int32_t act, void* dpre, void* dx,
                               void* dw, int32_t dw_f32, float* dbias, void* stream) {
  int st = check_sizes(rows, E, K, N, act, true);
  if (st != MOE_OK) return st;
  if (!expert_offsets || (dw_f32 != 0 && dw_f32 != 1)) return MOE_ERR_INVALID_ARG;
  const bool has_act = act != MOE_ACT_NONE;
  if (rows > 0) {
    if (!dy || (has_act && (!pre || !dpre)) || (dx && !w) || (dw && !x))
      return MOE_ERR_INVALID_ARG;
  }
  if (!aligned(dy, 16) || !aligned(pre, 16) || !aligned(x, 16) || !aligned(w, 16) ||
      !aligned(dpre, 16) || !aligned(dx, 16) || !aligned(dw, 16) || !aligned(dbias, 4) ||
      !aligned(expert_offsets, 4))
    return MOE_ERR_ALIGNMENT;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const void* d = has_act ? dpre : dy;
  const uint16_t* dyv = static_cast<const uint16_t*>(dy);
  const uint16_t* prev = static_cast<const uint16_t*>(pre);
  uint16_t* dprev = static_cast<uint16_t*>(dpre);
  with_act(act, [&](auto a) {
    if (dbias) {
      const auto sums = [&](auto kern, int threads, int cols) {
        return launch(kern, int64_t(E) * ((N + cols - 1) / cols), threads, s, dyv, prev,
                      expert_offsets, rows, E, N, dprev, dbias);
      };
      // Strips of 64 columns, of 256 threads where there are two a CU or few rows an expert (16 experts
      // of 1288 columns, 300 rows: 6.2 against 7.2 us with 1024), of 1024 where there are fewer; where
      // these would be under 64, strips of 16 columns.  Measured, gelu, in this order: 60
      // experts of 1024 columns (960 strips) 16384 rows 23 / 29 / 71 us, 256 of 2048 (8192) 1024 rows
      // 13 / 67 / 355, 8 of 7168 (896) 16384 rows 157 / 163 / 463, 8 of 1024 (128) 51 / 33 / 57, one of
      // 4096 (64) 8192 rows 180 / 108 / 106, one of 520 (9) 295 / 128 / 39.
      const int64_t strips = int64_t(E) * ((N + 63) / 64);
      st = strips >= 2 * kCus || rows <= int64_t(E) * 64 ? sums(pre_grad_kernel<a, 256, 64>, 256, 64)
           : strips >= 64     ? sums(pre_grad_kernel<a, 1024, 64>, 1024, 64)
                              : sums(pre_grad_kernel<a, 1024, 16>, 1024, 16);
    } else if (has_act && rows > 0) {
      st = launch(pre_kernel<a>, (rows * (N / 8) + 255) / 256, 256, s, dyv, prev, expert_offsets,
                  rows, E, N, dprev);
    }
  });
  if (st != MOE_OK) return st;
  return product_grads(d, x, expert_offsets, w, rows, E, N, K, dx, dw, dw_f32, s);
}

int moe_combine_backward(const void* dout, const void* y, const int32_t* pair_row,
                         const float* topk_w, int64_t T, int32_t H, int32_t k, int64_t capacity,
                         void* dy, float* dtopk_w, void* stream) {
  if (T < 0 || k < 1 || k > kMaxK || T > kMaxPairs / k || bad_features(H))
    return MOE_ERR_INVALID_ARG;
  if (H % 8 != 0) return MOE_ERR_ALIGNMENT;
  if (T == 0) return MOE_OK;
  if (!dout || !y || !pair_row || !topk_w || !dy || !dtopk_w) return MOE_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(pair_row, 4) ||
      !aligned(topk_w, 4) || !aligned(dtopk_w, 4))
    return MOE_ERR_ALIGNMENT;
  if (capacity < T * int64_t(k)) return MOE_ERR_CAPACITY;
  return launch(combine_grad_kernel, (T * k + 3) / 4, 256, static_cast<hipStream_t>(stream),
                static_cast<const u32x4*>(dout), static_cast<const u32x4*>(y), pair_row, topk_w, T,
                H / 8, k, capacity, static_cast<u32x4*>(dy), dtopk_w);
}

}  // extern "C"
