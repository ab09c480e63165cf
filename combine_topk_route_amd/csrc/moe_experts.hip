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

// 1 / (1 + exp(-z)); exp overflows to infinity for z < -88, which gives 0.
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

constexpr float kInvSqrt2 = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// z * Phi(z) through erfc, which keeps its relative precision in the left tail
// where 1 + erf cancels.
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_ACT_SILU: return z * sigmoid(z);
    case MOE_ACT_GELU: return 0.5f * z * erfcf(-z * kInvSqrt2);
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;  // a NaN stays one
    default: return z;
  }
}

// d act / dz (relu's is 0 at 0).
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_SILU: {
      const float s = sigmoid(z);
      return s * (1.f + z * (1.f - s));
    }
    case MOE_ACT_GELU:
      return 0.5f * erfcf(-z * kInvSqrt2) + z * expf(-0.5f * z * z) * kInvSqrt2Pi;
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    default: return 1.f;
  }
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

struct Tile {
  int e;         // expert, or -1 past the last tile
  int64_t row0;  // first row
  int rows;      // rows of this tile (1 .. BM)
  int nt;        // column tile
};

// Blocks are handed to the 8 XCDs in turn, and each XCD has an L2 of its own.
// So that the tiles an XCD works on at one time share their operands, tile
// numbers go to the XCDs in runs of `kRun` (its 32 CUs), or shorter ones where
// there are too few tiles to give each XCD a run.  A bijection on every 8 * kRun
// numbers; grids are rounded up to that.
constexpr int kXcds = 8, kRun = 32;

__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t total) {
  int run = kRun;
  while (run > 1 && total < int64_t(kXcds) * run) run >>= 1;
  const int64_t j = id / kXcds;
  return (j / run * kXcds + id % kXcds) * run + j % run;
}

// Tile `local` of a grid of mt x nt tiles: strips of 8 row tiles, inside a strip
// the row tile first, so that 32 neighbours read 8 + 4 strips of the operands.
__device__ __forceinline__ void grid_order(int64_t local, int64_t mt, int64_t nt, int64_t& m,
                                           int64_t& n) {
  const int64_t g = local / (8 * nt), rem = local - g * 8 * nt;
  const int64_t gm = mt - g * 8 < 8 ? mt - g * 8 : 8;
  m = g * 8 + rem % gm;
  n = rem / gm;
}

// The tile of block number `id`.  Every thread of the block calls it.
template <int BM, int THREADS>
__device__ Tile find_tile(const int32_t* off, int E, int64_t rows, int ncol, int64_t id) {
  __shared__ int64_t s_wave[THREADS / kWave];
  __shared__ Tile s_tile;
  const int per = (E + THREADS - 1) / THREADS;
  const int e0 = threadIdx.x * per;
  int64_t mine = 0;
  for (int i = 0; i < per && e0 + i < E; ++i) {
    int64_t lo, n;
    expert_rows(off, e0 + i, rows, lo, n);
    mine += (n + BM - 1) / BM;
  }
  int64_t incl = mine;
  for (int d = 1; d < kWave; d <<= 1) {
    const int64_t up = __shfl_up(incl, d);
    if (lane_id() >= d) incl += up;
  }
  const int w = threadIdx.x / kWave;
  if (threadIdx.x == 0) s_tile.e = -1;
  if (lane_id() == kWave - 1) s_wave[w] = incl;
  __syncthreads();
  int64_t pre = incl - mine, total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / kWave; ++i) {
    if (i < w) pre += s_wave[i];
    total += s_wave[i];
  }
  const int64_t seq = xcd_order(id, total * ncol);
  if (seq >= pre * ncol && seq < (pre + mine) * ncol) {
    for (int i = 0; i < per && e0 + i < E; ++i) {
      int64_t lo, n;
      expert_rows(off, e0 + i, rows, lo, n);
      const int64_t mt = (n + BM - 1) / BM;
      if (seq < (pre + mt) * ncol) {
        int64_t m, c;
        grid_order(seq - pre * ncol, mt, ncol, m, c);
        s_tile.e = e0 + i;
        s_tile.row0 = lo + m * BM;
        s_tile.rows = int(n - m * BM < BM ? n - m * BM : BM);
        s_tile.nt = int(c);
        break;
      }
      pre += mt;
    }
  }
  __syncthreads();
  Tile t = s_tile;
  __syncthreads();  // s_tile and s_wave may be written again
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  t.nt = __builtin_amdgcn_readfirstlane(t.nt);
  t.row0 = int64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(t.row0)))) |
           int64_t(__builtin_amdgcn_readfirstlane(int(t.row0 >> 32))) << 32;
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
//     of row r sits in slot c ^ swizzle(r), so that the 8 lanes that a 128-bit
//     read serves at once, rows apart by 128 bytes, find 8 different slots.
//   position contiguous: LDS row = k, R positions; read transposed
//     (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 values and each receives
//     one column).  Again the chunk order of a row depends on k, so that the 4
//     rows' pieces lie in different banks.
//
// Which position belongs to which row of the matrix instruction is free.  On the
// P side (PERM) row i of fragment f of a pair stands for position
// 8 (i / 4) + 4 f + i % 4 of 32, so that a lane's two fragments hold 8 consecutive
// positions and leave in one 16-byte store.

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
      : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
      : "m0");
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
template <bool KC_, bool PERM, int R, int W>
struct Side {
  static constexpr bool KC = KC_;
  static constexpr int kBytes = R * kBK * 2;
  static constexpr int kLoads = kBytes / 1024 / W;  // a wave's loads per stage
  static constexpr int kKRows = 512 / R;            // !KC: values of k in one load

  uint32_t voff[kLoads];
  const uint16_t* base;
  const uint16_t* base2;  // KC: base of the positions whose bit 5 is set (gated), or base
  int64_t ld;
  int64_t K;
  uint32_t bytes;  // KC: bytes of the valid rows;  else: bytes in front of the first column
  int kc;          // KC: this lane's k in the stage

  // `base` points at position 0, k 0.  KC: `valid` rows from there exist.  GATED: positions
  // 32 s + j, s odd, are row 16 (s - 1) + j behind `second`, s even those behind `base`.
  template <bool GATED>
  __device__ __forceinline__ void init(const uint16_t* first, const uint16_t* second, int64_t ld_,
                                       int64_t K_, int64_t valid) {
    base = first;
    base2 = second;
    ld = ld_;
    K = K_;
    const int w = wave_id(), l = lane_id();
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int t = j * W + w;
      if (KC) {
        const int r = t * 8 + l / 8;
        const int swz = PERM ? (r & 3) | ((r >> 1) & 4) : r & 7;
        const int c = (l % 8) ^ swz;
        kc = c * 8;  // the same for every j: W is even
        const int pos = GATED ? (r / 64) * 32 + r % 32 : r;
        voff[j] = uint32_t(pos) * uint32_t(ld * 2) + c * 16;
      } else {
        const int k = t * kKRows + l / (R / 8);
        const int g = PERM ? (k & 3) << 2 : (k & 3) << 1;
        voff[j] = uint32_t(k) * uint32_t(ld * 2) + ((l % (R / 8)) ^ g) * 16;
      }
    }
    if (KC)
      bytes = valid <= 0 ? 0u : uint32_t(valid < R ? valid : R) * uint32_t(ld * 2);
    else
      bytes = uint32_t(valid * 2);  // here `valid` is the first column's index in its row
  }

  // Start filling the stage at LDS address `lds` with k in [it * 64, it * 64 + 64).
  __device__ __forceinline__ void issue(uint32_t lds, int64_t it) const {
    const int w = wave_id();
    const int64_t k0 = it * kBK;
    if (KC) {
      const i32x4 r0 = resource(base, bytes);
      const i32x4 r1 = resource(base2, bytes);
      const bool whole = k0 + kBK <= K;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int t = j * W + w;
        const uint32_t v = whole || k0 + kc < K ? voff[j] : kOutside;
        load_to_lds(lds + t * 1024, v, (t >> 2) & 1 ? r1 : r0, whole ? int(k0 * 2) : (k0 < K ? int(k0 * 2) : 0));
      }
    } else {
      const int64_t rem = K - k0 < kBK ? K - k0 : kBK;
      const uint32_t n = rem <= 0 ? 0u : uint32_t(rem) * uint32_t(ld * 2) - bytes;
      const i32x4 r = resource(base + (rem <= 0 ? 0 : k0 * ld), n);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) load_to_lds(lds + (j * W + w) * 1024, voff[j], r, 0);
    }
  }
};

typedef __attribute__((address_space(3))) const bf16x8* LdsFrag;
typedef __attribute__((address_space(3))) s16x4* LdsTr;

__device__ __forceinline__ bf16x8 read_frag(uint32_t at) {
  return *reinterpret_cast<LdsFrag>(at);
}
// 4 values of k from `at`, the next 4 from `at` + 4 rows.
template <int ROW>
__device__ __forceinline__ bf16x8 read_frag_tr(uint32_t at) {
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<LdsTr>(at));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<LdsTr>(at + 4 * ROW));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The tile shape: BM x BN outputs by WM x WN waves, each (BM / WM) x 64, ST stages in LDS.
// A wave's row fragment i covers rows 16 (i * WM + wave row), so that a short tile loads every
// wave alike.
template <int BM_, int BN_, int WM_, int ST_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = BN_ / 64, ST = ST_;
  static constexpr int W = WM * WN, kThreads = W * kWave, MR = BM / WM / 16;
};

// acc[i][2 p + f] of MREP row fragments: position n = 64 wn + 32 p + 8 (lane / 16) + 4 f + 0..3
// against row m = 16 (i * WM + wm) + lane % 16.
template <typename S, int MREP, typename PS, typename QS>
__device__ __forceinline__ void product(f32x4 (&acc)[MREP][4], uint8_t* smem, const PS& P,
                                        const QS& Q, int64_t K) {
  static_assert(S::WM == 2, "the position-contiguous row offsets assume two wave rows");
  constexpr int kStage = PS::kBytes + QS::kBytes;
  constexpr int kLoads = PS::kLoads + QS::kLoads;
  constexpr int kPRow = S::BN * 2, kQRow = S::BM * 2;
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_address(smem));
  const int w = wave_id(), wm = w % S::WM, wn = w / S::WM;
  const int l = lane_id(), i = l % 16, q = l / 16;
#pragma unroll
  for (int a = 0; a < MREP; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  // where this lane reads, in a stage
  uint32_t pb[2], qb[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    pb[u] = PS::KC ? wn * 8192 + ((i / 4) * 8 + i % 4) * 128 +
                         (((u * 4 + q) ^ ((i & 3) | (i & 4))) * 16)
                   : (q * 8 + i / 4) * kPRow + (((wn * 8 + u * 4 + i % 4) ^ ((i / 4) << 2)) * 16);
    qb[u] = PS::kBytes +
            (QS::KC ? (wm * 16 + i) * 128 + (((u * 4 + q) ^ (i & 7)) * 16)
                    : (q * 8 + i / 4) * kQRow +
                          (((u * 4 + wm * 2 + (i % 4) / 2) ^ ((i / 4) << 1)) * 16) + (i & 1) * 8);
  }
  const int64_t n = (K + kBK - 1) / kBK;
  if (n == 0) return;
#pragma unroll
  for (int s = 0; s < S::ST - 1; ++s) {
    P.issue(lds + s * kStage, s);
    Q.issue(lds + s * kStage + PS::kBytes, s);
  }
  int cur = 0;
  for (int64_t it = 0; it < n; ++it) {
    stage_ready<(S::ST - 2) * kLoads>();
    const int to = cur == 0 ? S::ST - 1 : cur - 1;  // the stage read in the last step
    P.issue(lds + to * kStage, it + S::ST - 1);
    Q.issue(lds + to * kStage + PS::kBytes, it + S::ST - 1);
    const uint32_t at = lds + cur * kStage;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      bf16x8 p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        p[u] = PS::KC ? read_frag(at + pb[sub] + (u / 2) * 4096 + (u % 2) * 512)
                      : read_frag_tr<kPRow>(at + pb[u / 2] + sub * 32 * kPRow + (u % 2) * 8);
#pragma unroll
      for (int a = 0; a < MREP; ++a) {
        const bf16x8 qa =
            QS::KC ? read_frag(at + qb[sub] + a * 4096)
                   : read_frag_tr<kQRow>(at + qb[a & 1] + sub * 32 * kQRow + (a >> 1) * 128);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          acc[a][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[u], qa, acc[a][u], 0, 0, 0);
      }
    }
    cur = cur == S::ST - 1 ? 0 : cur + 1;
  }
  // loads still under way write zeros to LDS: they end before it is used again
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
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

__device__ __forceinline__ f32x4 act4(f32x4 v, int act) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = act_value(v[i], act);
  return v;
}

// The position of this lane's 8 values of pair p, and its row of fragment a, in the tile.
template <typename S>
__device__ __forceinline__ int lane_n(int p) {
  return wave_id() / S::WM * 64 + p * 32 + lane_id() / 16 * 8;
}
template <typename S>
__device__ __forceinline__ int lane_m(int a) {
  return (a * S::WM + wave_id() % S::WM) * 16 + lane_id() % 16;
}

// f<MREP>() with the fewest row fragments (a power of two) that cover `rows`: a tile at the end
// of an expert computes no more than twice its rows.
template <typename S, typename F>
__device__ __forceinline__ void by_height(int rows, F f) {
  const int need = (rows + 16 * S::WM - 1) / (16 * S::WM);
  if constexpr (S::MR >= 8)
    if (need > 4) return f(std::integral_constant<int, 8>{});
  if constexpr (S::MR >= 4)
    if (need > 2) return f(std::integral_constant<int, 4>{});
  if constexpr (S::MR >= 2)
    if (need > 1) return f(std::integral_constant<int, 2>{});
  f(std::integral_constant<int, 1>{});
}

template <typename S, bool PKC, bool QKC>
constexpr int lds_bytes() {
  return S::ST * (Side<PKC, true, S::BN, S::W>::kBytes + Side<QKC, false, S::BM, S::W>::kBytes);
}

// h = act(x Wg^T) * (x Wu^T): each wave's 64 positions are 32 gate columns and the same 32 up
// columns, so that one lane has both factors.
template <typename S>
__global__ __launch_bounds__(S::kThreads) void gated_kernel(
    const uint16_t* x, const int32_t* off, const uint16_t* w, int64_t rows, int E, int H, int I,
    int act, uint16_t* h, uint16_t* gu) {
  __shared__ __align__(1024) uint8_t smem[lds_bytes<S, true, true>()];
  constexpr int kCols = S::BN / 2;
  const int ncol = (I + kCols - 1) / kCols;
  for (int64_t id = blockIdx.x;; id += gridDim.x) {
    const Tile t = find_tile<S::BM, S::kThreads>(off, E, rows, ncol, id);
    if (t.e < 0) return;
    const int n0 = t.nt * kCols;
    const uint16_t* we = w + (int64_t(t.e) * 2 * I + n0) * H;
    Side<true, true, S::BN, S::W> P;
    Side<true, false, S::BM, S::W> Q;
    P.template init<true>(we, we + int64_t(I) * H, H, H, I - n0);
    const uint16_t* xe = x + t.row0 * H;
    Q.template init<false>(xe, xe, H, H, t.rows);
    by_height<S>(t.rows, [&](auto mrep) {
      constexpr int M = decltype(mrep)::value;
      f32x4 acc[M][4];
      product<S, M>(acc, smem, P, Q, H);
      const int n = n0 + wave_id() / S::WM * 32 + lane_id() / 16 * 8;
#pragma unroll
      for (int a = 0; a < M; ++a) {
        const int m = lane_m<S>(a);
        if (m >= t.rows || n >= I) continue;
        const int64_t row = t.row0 + m;
        store8(h + row * I + n, act4(acc[a][0], act) * acc[a][2], act4(acc[a][1], act) * acc[a][3]);
        if (gu != nullptr) {
          store8(gu + row * 2 * I + n, acc[a][0], acc[a][1]);
          store8(gu + row * 2 * I + I + n, acc[a][2], acc[a][3]);
        }
      }
    });
  }
}

// y = act(x W^T + bias) + residual, pre = act's argument.
template <typename S>
__global__ __launch_bounds__(S::kThreads) void matmul_kernel(
    const uint16_t* x, const int32_t* off, const uint16_t* w, const uint16_t* bias,
    const uint16_t* res, int64_t rows, int E, int K, int N, int act, uint16_t* y, uint16_t* pre) {
  __shared__ __align__(1024) uint8_t smem[lds_bytes<S, true, true>()];
  const int ncol = (N + S::BN - 1) / S::BN;
  for (int64_t id = blockIdx.x;; id += gridDim.x) {
    const Tile t = find_tile<S::BM, S::kThreads>(off, E, rows, ncol, id);
    if (t.e < 0) return;
    const int n0 = t.nt * S::BN;
    const uint16_t* we = w + (int64_t(t.e) * N + n0) * K;
    const uint16_t* xe = x + t.row0 * K;
    Side<true, true, S::BN, S::W> P;
    Side<true, false, S::BM, S::W> Q;
    P.template init<false>(we, we, K, K, N - n0);
    Q.template init<false>(xe, xe, K, K, t.rows);
    by_height<S>(t.rows, [&](auto mrep) {
      constexpr int M = decltype(mrep)::value;
      f32x4 acc[M][4];
      product<S, M>(acc, smem, P, Q, K);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int n = n0 + lane_n<S>(p);
        if (n >= N) continue;
        f32x4 b0 = {0.f, 0.f, 0.f, 0.f}, b1 = b0;
        if (bias != nullptr) load8(bias + int64_t(t.e) * N + n, b0, b1);
#pragma unroll
        for (int a = 0; a < M; ++a) {
          const int m = lane_m<S>(a);
          if (m >= t.rows) continue;
          const int64_t at = (t.row0 + m) * N + n;
          f32x4 v0 = acc[a][2 * p] + b0, v1 = acc[a][2 * p + 1] + b1;
          if (pre != nullptr) store8(pre + at, v0, v1);
          v0 = act4(v0, act);
          v1 = act4(v1, act);
          if (res != nullptr) {
            f32x4 r0, r1;
            load8(res + at, r0, r1);
            v0 += r0;
            v1 += r1;
          }
          store8(y + at, v0, v1);
        }
      }
    });
  }
}

// dx = d W: the weights [N, K] are contiguous along the output's own index.
template <typename S>
__global__ __launch_bounds__(S::kThreads) void data_grad_kernel(
    const uint16_t* d, const int32_t* off, const uint16_t* w, int64_t rows, int E, int N, int K,
    uint16_t* dx) {
  __shared__ __align__(1024) uint8_t smem[lds_bytes<S, false, true>()];
  const int ncol = (K + S::BN - 1) / S::BN;
  for (int64_t id = blockIdx.x;; id += gridDim.x) {
    const Tile t = find_tile<S::BM, S::kThreads>(off, E, rows, ncol, id);
    if (t.e < 0) return;
    const int n0 = t.nt * S::BN;
    const uint16_t* we = w + int64_t(t.e) * N * K + n0;
    const uint16_t* de = d + t.row0 * N;
    Side<false, true, S::BN, S::W> P;
    Side<true, false, S::BM, S::W> Q;
    P.template init<false>(we, we, K, N, n0);
    Q.template init<false>(de, de, N, N, t.rows);
    by_height<S>(t.rows, [&](auto mrep) {
      constexpr int M = decltype(mrep)::value;
      f32x4 acc[M][4];
      product<S, M>(acc, smem, P, Q, N);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int n = n0 + lane_n<S>(p);
#pragma unroll
        for (int a = 0; a < M; ++a) {
          const int m = lane_m<S>(a);
          if (m < t.rows && n < K)
            store8(dx + (t.row0 + m) * K + n, acc[a][2 * p], acc[a][2 * p + 1]);
        }
      }
    });
  }
}

// dW[e] = d^T x over the expert's rows: both sides are contiguous along the
// output's indexes.  An expert without rows gets zeros.
template <typename S, bool F32>
__global__ __launch_bounds__(S::kThreads) void weight_grad_kernel(
    const uint16_t* d, const uint16_t* x, const int32_t* off, int64_t rows, int E, int N, int K,
    void* dw) {
  __shared__ __align__(1024) uint8_t smem[lds_bytes<S, false, false>()];
  const int64_t nn = (N + S::BM - 1) / S::BM, nk = (K + S::BN - 1) / S::BN;
  const int64_t total = E * nn * nk;
  for (int64_t id = blockIdx.x;; id += gridDim.x) {
    const int64_t seq = xcd_order(id, total);
    if (seq >= total) return;
    const int e = int(seq / (nn * nk));
    int64_t mt, ct;
    grid_order(seq - e * nn * nk, nn, nk, mt, ct);
    const int m0 = int(mt) * S::BM, n0 = int(ct) * S::BN;
    int64_t lo, cnt;
    expert_rows(off, e, rows, lo, cnt);
    const uint16_t* xe = x + lo * K + n0;
    const uint16_t* de = d + lo * N + m0;
    Side<false, true, S::BN, S::W> P;
    Side<false, false, S::BM, S::W> Q;
    P.template init<false>(xe, xe, K, cnt, n0);
    Q.template init<false>(de, de, N, cnt, m0);
    f32x4 acc[S::MR][4];
    product<S, S::MR>(acc, smem, P, Q, cnt);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int n = n0 + lane_n<S>(p);
#pragma unroll
      for (int a = 0; a < S::MR; ++a) {
        const int m = m0 + lane_m<S>(a);
        if (m >= N || n >= K) continue;
        const int64_t at = (int64_t(e) * N + m) * K + n;
        if (F32) {
          f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(dw) + at);
          o[0] = acc[a][2 * p];
          o[1] = acc[a][2 * p + 1];
        } else {
          store8(static_cast<uint16_t*>(dw) + at, acc[a][2 * p], acc[a][2 * p + 1]);
        }
      }
    }
    __syncthreads();  // every wave has read its last stage before the next tile fills it
  }
}

// ---------------------------------------------------------------------------
// elementwise gradients
// ---------------------------------------------------------------------------

// [dg du] from dh and the kept factors, 8 columns per thread.
__global__ __launch_bounds__(256) void gated_grad_kernel(const uint16_t* dh, const uint16_t* gu,
                                                         const int32_t* off, int64_t rows, int E,
                                                         int I, int act, uint16_t* dgu) {
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
      og[q] = pack_bf16x2(h0 * bf16_lo(vu[q]) * act_slope(g0, act),
                          h1 * bf16_hi(vu[q]) * act_slope(g1, act));
      ou[q] = pack_bf16x2(h0 * act_value(g0, act), h1 * act_value(g1, act));
    }
    *reinterpret_cast<u32x4*>(dgu + row * 2 * I + c) = og;
    *reinterpret_cast<u32x4*>(dgu + row * 2 * I + I + c) = ou;
  }
}

// dpre = dy * act'(pre) and dbias[e] = its sum over the expert's rows, in a
// fixed order: a block owns 64 columns of one expert, 32 threads a column
// chunk, each adding every 32nd row.
__global__ __launch_bounds__(256) void pre_grad_kernel(const uint16_t* dy, const uint16_t* pre,
                                                       const int32_t* off, int64_t rows, int E,
                                                       int N, int act, uint16_t* dpre,
                                                       float* dbias) {
  __shared__ float part[32][65];
  const int64_t strips = (N + 63) / 64;
  for (int64_t u = blockIdx.x; u < E * strips; u += gridDim.x) {
    const int e = int(u / strips);
    const int c = int(u % strips) * 64 + (threadIdx.x % 8) * 8;
    int64_t lo, cnt;
    expert_rows(off, e, rows, lo, cnt);
    float sum[8] = {};
    if (c < N) {
      for (int64_t r = threadIdx.x / 8; r < cnt; r += 32) {
        const int64_t at = (lo + r) * N + c;
        const u32x4 vy = *reinterpret_cast<const u32x4*>(dy + at);
        u32x4 vp = {0u, 0u, 0u, 0u}, o;
        if (act != MOE_ACT_NONE) vp = *reinterpret_cast<const u32x4*>(pre + at);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float d0 = bf16_lo(vy[q]) * act_slope(bf16_lo(vp[q]), act);
          const float d1 = bf16_hi(vy[q]) * act_slope(bf16_hi(vp[q]), act);
          sum[2 * q] += d0;
          sum[2 * q + 1] += d1;
          o[q] = pack_bf16x2(d0, d1);
        }
        if (dpre != nullptr) *reinterpret_cast<u32x4*>(dpre + at) = o;
      }
    }
    if (dbias == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 8; ++q) part[threadIdx.x / 8][(threadIdx.x % 8) * 8 + q] = sum[q];
    __syncthreads();
    const int64_t col = (u % strips) * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < N) {
      float s = 0.f;
      for (int r = 0; r < 32; ++r) s += part[r][threadIdx.x];
      dbias[int64_t(e) * N + col] = s;
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

// The sizes every product shares; MOE_OK with rows == 0 allowed.
int check_sizes(int64_t rows, int32_t E, int32_t a, int32_t b, int32_t act, bool none_ok) {
  if (rows < 0 || rows > kMaxPairs || E < 1 || E > kMaxE) return MOE_ERR_INVALID_ARG;
  if (bad_features(a) || bad_features(b)) return MOE_ERR_INVALID_ARG;
  if (act < (none_ok ? MOE_ACT_NONE : MOE_ACT_SILU) || act > MOE_ACT_RELU)
    return MOE_ERR_INVALID_ARG;
  if (a % 8 != 0 || b % 8 != 0) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Blocks for tiles of at most `bm` rows that `rows` rows in E runs can need, `cols` to a row of
// tiles, rounded up to what xcd_order permutes.
int64_t row_tile_blocks(int64_t rows, int32_t E, int bm, int64_t cols) {
  const int64_t runs = rows < E ? rows : E;
  const int64_t n = (rows / bm + runs) * cols, group = int64_t(kXcds) * kRun;
  return (n + group - 1) / group * group;
}

// Whether the experts have too few rows each for the tall tiles.
bool few_rows(int64_t rows, int32_t E) { return rows <= int64_t(E) * 32; }

using Big = Shape<256, 256, 2, 2>;    // 128 KiB of LDS, one block of 8 waves a CU
using Small = Shape<64, 128, 2, 4>;   // 96 KiB, 4 waves

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
  auto run = [&](auto shape, auto kern) {
    using S = decltype(shape);
    return launch(kern, row_tile_blocks(rows, E, S::BM, (I + S::BN / 2 - 1) / (S::BN / 2)),
                  S::kThreads, static_cast<hipStream_t>(stream),
                  static_cast<const uint16_t*>(x), expert_offsets,
                  static_cast<const uint16_t*>(w_gate_up), rows, E, H, I, act,
                  static_cast<uint16_t*>(h), static_cast<uint16_t*>(gate_up));
  };
  return few_rows(rows, E) ? run(Small{}, gated_kernel<Small>) : run(Big{}, gated_kernel<Big>);
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
  auto run = [&](auto shape, auto kern) {
    using S = decltype(shape);
    return launch(kern, row_tile_blocks(rows, E, S::BM, (N + S::BN - 1) / S::BN), S::kThreads,
                  static_cast<hipStream_t>(stream), static_cast<const uint16_t*>(x),
                  expert_offsets, static_cast<const uint16_t*>(w),
                  static_cast<const uint16_t*>(bias), static_cast<const uint16_t*>(residual), rows,
                  E, K, N, act, static_cast<uint16_t*>(y), static_cast<uint16_t*>(pre));
  };
  return few_rows(rows, E) ? run(Small{}, matmul_kernel<Small>) : run(Big{}, matmul_kernel<Big>);
}

static int weight_grad(const void* d, const void* x, const int32_t* off, int64_t rows, int E,
                       int N, int K, void* dw, int dw_f32, hipStream_t s) {
  const int64_t n = int64_t(E) * ((N + Big::BM - 1) / Big::BM) * ((K + Big::BN - 1) / Big::BN);
  const int64_t group = int64_t(kXcds) * kRun;
  return launch(dw_f32 ? weight_grad_kernel<Big, true> : weight_grad_kernel<Big, false>,
                (n + group - 1) / group * group, Big::kThreads, s,
                static_cast<const uint16_t*>(d), static_cast<const uint16_t*>(x), off, rows, E, N,
                K, dw);
}

static int data_grad(const void* d, const int32_t* off, const void* w, int64_t rows, int E, int N,
                     int K, void* dx, hipStream_t s) {
  return launch(data_grad_kernel<Big>,
                row_tile_blocks(rows, E, Big::BM, (K + Big::BN - 1) / Big::BN), Big::kThreads, s,
                static_cast<const uint16_t*>(d), off, static_cast<const uint16_t*>(w), rows, E, N,
                K, static_cast<uint16_t*>(dx));
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
    st = launch(gated_grad_kernel, (rows * (I / 8) + 255) / 256, 256, s,
                static_cast<const uint16_t*>(dh), static_cast<const uint16_t*>(gate_up),
                expert_offsets, rows, E, I, act, static_cast<uint16_t*>(dgate_up));
    if (st == MOE_OK && dx)
      st = data_grad(dgate_up, expert_offsets, w_gate_up, rows, E, 2 * I, H, dx, s);
  }
  if (st == MOE_OK && dw)
    st = weight_grad(dgate_up, x, expert_offsets, rows, E, 2 * I, H, dw, dw_f32, s);
  return st;
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
  if ((has_act && rows > 0) || dbias) {
    st = launch(pre_grad_kernel, int64_t(E) * ((N + 63) / 64), 256, s,
                static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(pre),
                expert_offsets, rows, E, N, act,
                has_act ? static_cast<uint16_t*>(dpre) : nullptr, dbias);
  }
  if (st == MOE_OK && dx && rows > 0) st = data_grad(d, expert_offsets, w, rows, E, N, K, dx, s);
  if (st == MOE_OK && dw) st = weight_grad(d, x, expert_offsets, rows, E, N, K, dw, dw_f32, s);
  return st;
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
