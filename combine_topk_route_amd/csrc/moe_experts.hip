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

// The tile with index `seq` in the order expert, column tile, row tile (the
// row tiles of one expert that share a strip of weights are neighbours).
// Every thread of the block calls it; blockDim.x >= 256.
template <int BM>
__device__ Tile find_tile(const int32_t* off, int E, int64_t rows, int ncol, int64_t seq) {
  __shared__ int64_t s_wave[16];
  __shared__ Tile s_tile;
  const int per = (E + blockDim.x - 1) / blockDim.x;
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
  int64_t pre = incl - mine;
  for (int i = 0; i < w; ++i) pre += s_wave[i];
  if (seq >= pre * ncol && seq < (pre + mine) * ncol) {
    for (int i = 0; i < per && e0 + i < E; ++i) {
      int64_t lo, n;
      expert_rows(off, e0 + i, rows, lo, n);
      const int64_t mt = (n + BM - 1) / BM;
      if (seq < (pre + mt) * ncol) {
        const int64_t local = seq - pre * ncol;
        const int64_t m = local % mt;
        s_tile.e = e0 + i;
        s_tile.row0 = lo + m * BM;
        s_tile.rows = int(n - m * BM < BM ? n - m * BM : BM);
        s_tile.nt = int(local / mt);
        break;
      }
      pre += mt;
    }
  }
  __syncthreads();
  const Tile t = s_tile;
  __syncthreads();  // s_tile and s_wave may be written again
  return t;
}

// ---------------------------------------------------------------------------
// the product of one 64 x 64 tile
// ---------------------------------------------------------------------------

// One side of the product: `at(i)` is the position of tile index i along the
// side's own dimension, or -1 outside it.
//   KC: element (i, k) = base[at(i) * ld + k]     (k contiguous)
//   else element (i, k) = base[k * ld + at(i)]    (i contiguous)
constexpr int kTile = 64, kBK = 32, kPad = 8;

template <bool KC, typename At>
__device__ __forceinline__ void stage(uint16_t (*s)[kBK + kPad], const uint16_t* base, int64_t ld,
                                      int64_t k0, int64_t K, At at) {
  // 64 x 32 elements = 256 chunks of 8, one per thread
  const int t = threadIdx.x;
  if (KC) {
    const int i = t / 4, k = (t % 4) * 8;
    const int64_t p = at(i);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (p >= 0 && k0 + k < K) v = *reinterpret_cast<const u32x4*>(base + p * ld + k0 + k);
    *reinterpret_cast<u32x4*>(&s[i][k]) = v;
  } else {
    const int k = t / 8, i = (t % 8) * 8;
    const int64_t p = at(i);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (p >= 0 && k0 + k < K) v = *reinterpret_cast<const u32x4*>(base + (k0 + k) * ld + p);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      s[i + 2 * q][k] = uint16_t(v[q]);
      s[i + 2 * q + 1][k] = uint16_t(v[q] >> 16);
    }
  }
}

// acc[a][b]: P rows 16 a + (lane / 16) * 4 + 0..3 against Q row 16 b + lane % 16,
// of this wave's 32 x 32 quarter.
template <bool PKC, bool QKC, typename PAt, typename QAt>
__device__ __forceinline__ void product(f32x4 (&acc)[2][2], const uint16_t* P, int64_t ldp,
                                        PAt pat, const uint16_t* Q, int64_t ldq, QAt qat,
                                        int64_t K) {
  __shared__ __align__(16) uint16_t sp[kTile][kBK + kPad];
  __shared__ __align__(16) uint16_t sq[kTile][kBK + kPad];
  const int w = threadIdx.x / kWave, wp = w / 2, wq = w % 2;
  const int r = lane_id() % 16, kk = (lane_id() / 16) * 8;
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t k0 = 0; k0 < K; k0 += kBK) {
    stage<PKC>(sp, P, ldp, k0, K, pat);
    stage<QKC>(sq, Q, ldq, k0, K, qat);
    __syncthreads();
    bf16x8 p[2], q[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      p[a] = *reinterpret_cast<const bf16x8*>(&sp[wp * 16 + a * 32 + r][kk]);
      q[a] = *reinterpret_cast<const bf16x8*>(&sq[wq * 32 + a * 16 + r][kk]);
    }
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[a], q[b], acc[a][b], 0, 0, 0);
    __syncthreads();
  }
}

// Tile index along P of this lane's first accumulator of block a, and along Q
// of block b.
__device__ __forceinline__ int lane_p(int a) {
  return (threadIdx.x / kWave / 2) * 16 + a * 32 + (lane_id() / 16) * 4;
}
__device__ __forceinline__ int lane_q(int b) {
  return (threadIdx.x / kWave % 2) * 32 + b * 16 + lane_id() % 16;
}

__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  const u32x2 v = *reinterpret_cast<const u32x2*>(p);
  return f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
}

// h = act(x Wg^T) * (x Wu^T): a tile holds 32 gate columns and the same 32 up
// columns, 16 apart in the waves' order, so that one lane has both factors.
__global__ __launch_bounds__(256) void gated_kernel(const uint16_t* x, const int32_t* off,
                                                    const uint16_t* w, int64_t rows, int E, int H,
                                                    int I, int act, uint16_t* h, uint16_t* gu) {
  const int ncol = (I + 31) / 32;
  for (int64_t seq = blockIdx.x;; seq += gridDim.x) {
    const Tile t = find_tile<kTile>(off, E, rows, ncol, seq);
    if (t.e < 0) return;
    f32x4 acc[2][2];
    product<true, true>(
        acc, w + int64_t(t.e) * 2 * I * H, H,
        [&](int i) -> int64_t {
          const int n = t.nt * 32 + i % 32;
          return n < I ? n + (i / 32) * int64_t(I) : -1;
        },
        x + t.row0 * H, H, [&](int i) -> int64_t { return i < t.rows ? i : -1; }, H);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int q = lane_q(b), n = t.nt * 32 + lane_p(0);
      if (q >= t.rows || n >= I) continue;
      const int64_t row = t.row0 + q;
      f32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = act_value(acc[0][b][i], act) * acc[1][b][i];
      store4(h + row * I + n, v);
      if (gu != nullptr) {
        store4(gu + row * 2 * I + n, acc[0][b]);
        store4(gu + row * 2 * I + I + n, acc[1][b]);
      }
    }
  }
}

// y = act(x W^T + bias) + residual, pre = act's argument.
__global__ __launch_bounds__(256) void matmul_kernel(const uint16_t* x, const int32_t* off,
                                                     const uint16_t* w, const uint16_t* bias,
                                                     const uint16_t* res, int64_t rows, int E,
                                                     int K, int N, int act, uint16_t* y,
                                                     uint16_t* pre) {
  const int ncol = (N + kTile - 1) / kTile;
  for (int64_t seq = blockIdx.x;; seq += gridDim.x) {
    const Tile t = find_tile<kTile>(off, E, rows, ncol, seq);
    if (t.e < 0) return;
    f32x4 acc[2][2];
    product<true, true>(
        acc, w + int64_t(t.e) * N * K, K,
        [&](int i) -> int64_t { return t.nt * kTile + i < N ? t.nt * kTile + i : -1; },
        x + t.row0 * K, K, [&](int i) -> int64_t { return i < t.rows ? i : -1; }, K);
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int q = lane_q(b), n = t.nt * kTile + lane_p(a);
        if (q >= t.rows || n >= N) continue;
        const int64_t at = (t.row0 + q) * N + n;
        f32x4 v = acc[a][b];
        if (bias != nullptr) v += load4(bias + int64_t(t.e) * N + n);
        if (pre != nullptr) store4(pre + at, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = act_value(v[i], act);
        if (res != nullptr) v += load4(res + at);
        store4(y + at, v);
      }
  }
}

// dx = d W: the weights [N, K] are contiguous along the output's own index.
__global__ __launch_bounds__(256) void data_grad_kernel(const uint16_t* d, const int32_t* off,
                                                        const uint16_t* w, int64_t rows, int E,
                                                        int N, int K, uint16_t* dx) {
  const int ncol = (K + kTile - 1) / kTile;
  for (int64_t seq = blockIdx.x;; seq += gridDim.x) {
    const Tile t = find_tile<kTile>(off, E, rows, ncol, seq);
    if (t.e < 0) return;
    f32x4 acc[2][2];
    product<false, true>(
        acc, w + int64_t(t.e) * N * K, K,
        [&](int i) -> int64_t { return t.nt * kTile + i < K ? t.nt * kTile + i : -1; },
        d + t.row0 * N, N, [&](int i) -> int64_t { return i < t.rows ? i : -1; }, N);
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int q = lane_q(b), n = t.nt * kTile + lane_p(a);
        if (q < t.rows && n < K) store4(dx + (t.row0 + q) * K + n, acc[a][b]);
      }
  }
}

// dW[e] = d^T x over the expert's rows: both sides are contiguous along the
// output's indexes.  An expert without rows gets zeros.
template <bool F32>
__global__ __launch_bounds__(256) void weight_grad_kernel(const uint16_t* d, const uint16_t* x,
                                                          const int32_t* off, int64_t rows, int E,
                                                          int N, int K, void* dw) {
  const int64_t nn = (N + kTile - 1) / kTile, nk = (K + kTile - 1) / kTile;
  for (int64_t seq = blockIdx.x; seq < E * nn * nk; seq += gridDim.x) {
    const int e = int(seq / (nn * nk));
    const int n0 = int(seq % (nn * nk) / nk) * kTile, c0 = int(seq % nk) * kTile;
    int64_t lo, cnt;
    expert_rows(off, e, rows, lo, cnt);
    f32x4 acc[2][2];
    product<false, false>(
        acc, x + lo * K, K, [&](int i) -> int64_t { return c0 + i < K ? c0 + i : -1; },
        d + lo * N, N, [&](int i) -> int64_t { return n0 + i < N ? n0 + i : -1; }, cnt);
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int n = n0 + lane_q(b), c = c0 + lane_p(a);
        if (n >= N || c >= K) continue;
        const int64_t at = (int64_t(e) * N + n) * K + c;
        if (F32)
          *reinterpret_cast<f32x4*>(static_cast<float*>(dw) + at) = acc[a][b];
        else
          store4(static_cast<uint16_t*>(dw) + at, acc[a][b]);
      }
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

// Tiles of at most `bm` rows that `rows` rows in E runs can need.
int64_t most_row_tiles(int64_t rows, int32_t E, int bm) {
  const int64_t runs = rows < E ? rows : E;
  return rows / bm + runs;
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
  const int64_t blocks = most_row_tiles(rows, E, kTile) * ((I + 31) / 32);
  return launch(gated_kernel, blocks, 256, static_cast<hipStream_t>(stream),
                static_cast<const uint16_t*>(x), expert_offsets,
                static_cast<const uint16_t*>(w_gate_up), rows, E, H, I, act,
                static_cast<uint16_t*>(h), static_cast<uint16_t*>(gate_up));
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
  const int64_t blocks = most_row_tiles(rows, E, kTile) * ((N + kTile - 1) / kTile);
  return launch(matmul_kernel, blocks, 256, static_cast<hipStream_t>(stream),
                static_cast<const uint16_t*>(x), expert_offsets, static_cast<const uint16_t*>(w),
                static_cast<const uint16_t*>(bias), static_cast<const uint16_t*>(residual), rows,
                E, K, N, act, static_cast<uint16_t*>(y), static_cast<uint16_t*>(pre));
}

static int weight_grad(const void* d, const void* x, const int32_t* off, int64_t rows, int E,
                       int N, int K, void* dw, int dw_f32, hipStream_t s) {
  const int64_t blocks =
      int64_t(E) * ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile);
  return launch(dw_f32 ? weight_grad_kernel<true> : weight_grad_kernel<false>, blocks, 256, s,
                static_cast<const uint16_t*>(d), static_cast<const uint16_t*>(x), off, rows, E, N,
                K, dw);
}

static int data_grad(const void* d, const int32_t* off, const void* w, int64_t rows, int E, int N,
                     int K, void* dx, hipStream_t s) {
  const int64_t blocks = most_row_tiles(rows, E, kTile) * ((K + kTile - 1) / kTile);
  return launch(data_grad_kernel, blocks, 256, s, static_cast<const uint16_t*>(d), off,
                static_cast<const uint16_t*>(w), rows, E, N, K, static_cast<uint16_t*>(dx));
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
