// The MX4 linear layer at few tokens (M <= 64):
//     Y [M, N] = Q(X) W^T + T B^T,   T = bf16(scale X A^T)
// The weight's bytes bound it, then the latency of a launch's few loads, so W
// goes from memory straight into registers, every wave issues the loads of a
// pass before the first product, and there are two launches at most.
//
// k_mx4_prep: partial sums P of X A^T, one workgroup per (slice of the
//   columns, 16 adapter rows, 16 tokens); its 16 waves split the slice and are
//   summed in LDS in wave order.  Further workgroups of the same launch round
//   X to MX4.  With k_mx4_sum it also serves more tokens, ahead of the tiles.
// k_mx4_small: one workgroup per 16 weight rows, its waves take slabs of 256
//   columns in turn: v_mfma_scale_f32_16x16x128 with W as the left operand
//   (lane l: row l % 16, block l / 16 of 128 columns) and 16 tokens a product
//   as the right one.  The waves' sums meet in LDS in wave order; T B^T is
//   added there, T from the partials' sum.  Without a LoRA pair and with few
//   workgroups a lane rounds the block of X that it supplies itself, 32 bf16
//   of one token: the block's maximum needs no other lane.
//
// r = 64: 1 x 11008 x 4096 takes 4.2 + 7.7 us in a kernel trace (W's 24 MB at 3.1
// TB/s; 4.3 + 6.7 by torch's profiler, whose figures stand beside the rules
// below), 64 x 4096 x 11008 5 + 21 us.
#include <algorithm>

#include "common.h"
#include "launch.h"
#include "tile.h"

namespace qlora {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

constexpr int kPrepWaves = 16;
// Columns of a slice of the partial sums: 32 a step, two steps a wave.  A
// compute unit fetches some 30 KB/us, so many small workgroups make them: at 32
// to 64 tokens of 4096 columns 4.4 us, with four steps a wave 6.0.  The main
// kernel then sums twice the slices, which costs it as much only at 64 tokens
// of 11008 columns (25.7 us in all against 25.2).
constexpr int kSteps = 2;
constexpr int kSlice = kPrepWaves * 32 * kSteps;
constexpr int kMainRows = 16;         // weight rows of a workgroup
constexpr int kFusedTokens = 16;      // see fused_ok
constexpr int kFusedGrid = 256;

struct SmallArgs {
  const uint16_t *X;                  // [M, K] bf16 (fused)
  const uint8_t *xc, *xs;             // X in MX4 (otherwise)
  const uint8_t *wc, *ws;
  const uint16_t *A, *B;
  const uint16_t *T;                  // T given, or null: from P
  float *P;                           // [S][M][r]
  uint16_t *Y, *Tout;
  int M, N, K, r;
  int S, slice;                       // column slices of P
  float scale;
};

__device__ __forceinline__ i32x8_t widen(i32x4_t v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }

// 8 bf16 of a row of length len from column j on, zero past it.
__device__ __forceinline__ bf16x8_t load8(const uint16_t *row, int j, int len, bool vec) {
  if (vec) return j < len ? *reinterpret_cast<const bf16x8_t *>(row + j) : bf16x8_t{};
  uint16_t v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = j + e < len ? row[j + e] : static_cast<uint16_t>(0);
  return __builtin_bit_cast(bf16x8_t, v);
}

// A block of 32 bf16 in MX4: codes and scale byte, by the codec's rules.
__device__ __forceinline__ uint32_t round_block(const uint32_t (&x)[16], i32x4_t &codes) {
  u16x2_t top = {0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, x[i] & 0x7FFF7FFFu));
  const uint32_t e = static_cast<uint32_t>(max(top[0], top[1])) >> 7;
  const uint32_t byte = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
  const float f = mx4_scale(byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x[4 * i]), f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x[4 * i + 1]), f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x[4 * i + 2]), f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x[4 * i + 3]), f, 3);
    codes[i] = byte == 255u ? 0 : static_cast<int>(c);
  }
  return byte;
}

}  // namespace

// A wave's steps are all loaded before the first product.  Workgroups from
// `downs` on round X.
__global__ __launch_bounds__(kPrepWaves * 64) void k_mx4_prep(const SmallArgs a, int downs, uint8_t *xc, uint8_t *xs) {
  __shared__ float red[kPrepWaves][256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (static_cast<int>(blockIdx.x) >= downs) {
    // A block of X a thread; 8 threads a slab of a row.
    const int slabs = (a.K + 255) / 256;
    const int64_t id = static_cast<int64_t>(blockIdx.x - downs) * (kPrepWaves * 64) + threadIdx.x;
    const int64_t rs = id >> 3;
    const int b = static_cast<int>(id & 7);
    const int row = static_cast<int>(rs / slabs), slab = static_cast<int>(rs % slabs);
    if (row >= a.M) return;
    const int k = slab * 256 + b * 32;
    i32x4_t codes = {0, 0, 0, 0};
    uint32_t byte = 0;
    if (k < a.K) {
      uint32_t x[16];
      const uint4 *p = reinterpret_cast<const uint4 *>(a.X + static_cast<int64_t>(row) * a.K + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = p[i];
        x[4 * i] = v.x;
        x[4 * i + 1] = v.y;
        x[4 * i + 2] = v.z;
        x[4 * i + 3] = v.w;
      }
      byte = round_block(x, codes);
    }
    *reinterpret_cast<i32x4_t *>(xc + (static_cast<int64_t>(row) * slabs + slab) * 128 + b * 16) = codes;
    xs[(static_cast<int64_t>(slab) * a.M + row) * 8 + b] = static_cast<uint8_t>(byte);
    return;
  }
  const int jts = (a.r + 15) / 16, mts = (a.M + 15) / 16;
  const int jt = blockIdx.x % jts, mt = blockIdx.x / jts % mts, s = blockIdx.x / (jts * mts);
  const int nl = lane & 15, g = lane >> 4;
  const int k0 = s * a.slice + wave * (32 * kSteps);
  const uint16_t *ar = a.A + static_cast<int64_t>(min(16 * jt + nl, a.r - 1)) * a.K;
  const uint16_t *xr = a.X + static_cast<int64_t>(min(16 * mt + nl, a.M - 1)) * a.K;
  bf16x8_t av[kSteps], xv[kSteps];
#pragma unroll
  for (int h = 0; h < kSteps; ++h) {
    const int c = min(k0 + 32 * h, a.K - 32) + 8 * g;   // K % 32 == 0: a step is whole or absent
    av[h] = *reinterpret_cast<const bf16x8_t *>(ar + c);
    xv[h] = *reinterpret_cast<const bf16x8_t *>(xr + c);
  }
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < kSteps; ++h)
    if (k0 + 32 * h < a.K) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[h], xv[h], acc, 0, 0, 0);
  *reinterpret_cast<f32x4_t *>(&red[wave][4 * lane]) = acc;   // adapter rows 4 (l / 16) + e of token l % 16
  __syncthreads();
  if (threadIdx.x >= 256) return;
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kPrepWaves; ++w) v += red[w][threadIdx.x];
  const int l = threadIdx.x >> 2, e = threadIdx.x & 3;
  const int j = 16 * jt + 4 * (l >> 4) + e, m = 16 * mt + (l & 15);
  if (j < a.r && m < a.M) a.P[(static_cast<int64_t>(s) * a.M + m) * a.r + j] = v;
}

namespace {

// What a wave loads for a slab.
template <int kMB, bool kFused>
struct Pass {
  i32x4_t w[2];
  uint2 wb;
  i32x4_t x[kMB][2];       // not fused
  uint2 xb[kMB];
  uint32_t raw[2][16];     // fused
};

// T [M, r] as bf16 into LDS, zero up to the next 32 columns: given, or the
// scaled sum of the partials, kPlanes slices' loads at a time.
template <int kMB, int kThreads, int kPlanes>
__device__ __forceinline__ void put_T(const SmallArgs &a, uint16_t (*sT)[136]) {
  const int rp = (a.r + 31) / 32 * 32, quads = rp / 4;
  const bool vec = (a.r & 3) == 0;
  for (int i = threadIdx.x; i < 16 * kMB * quads; i += kThreads) {
    const int m = i / quads, j = 4 * (i - m * quads);
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    uint16_t v[4] = {0, 0, 0, 0};
    if (m < a.M && j < a.r) {
      if (a.T && (a.r & 3) == 0) {
        const uint2 q = *reinterpret_cast<const uint2 *>(a.T + static_cast<int64_t>(m) * a.r + j);
        v[0] = static_cast<uint16_t>(q.x);
        v[1] = static_cast<uint16_t>(q.x >> 16);
        v[2] = static_cast<uint16_t>(q.y);
        v[3] = static_cast<uint16_t>(q.y >> 16);
      } else if (a.T) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < a.r) v[e] = a.T[static_cast<int64_t>(m) * a.r + j + e];
      } else {
        const float *p = a.P + static_cast<int64_t>(m) * a.r + j;
        const int64_t plane = static_cast<int64_t>(a.M) * a.r;
        for (int s0 = 0; s0 < a.S; s0 += kPlanes) {
          float q[kPlanes][4];
#pragma unroll
          for (int s = 0; s < kPlanes; ++s) {
            const float *ps = p + plane * min(s0 + s, a.S - 1);
            if (vec) {
              const float4 f = *reinterpret_cast<const float4 *>(ps);
              q[s][0] = f.x;
              q[s][1] = f.y;
              q[s][2] = f.z;
              q[s][3] = f.w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) q[s][e] = j + e < a.r ? ps[e] : 0.f;
            }
          }
#pragma unroll
          for (int s = 0; s < kPlanes; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] += s0 + s < a.S ? q[s][e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = f32_to_bf16(a.scale * t[e]);
          if (blockIdx.x == 0 && a.Tout && j + e < a.r) a.Tout[static_cast<int64_t>(m) * a.r + j + e] = v[e];
        }
      }
    }
    *reinterpret_cast<uint2 *>(&sT[m][j]) = make_uint2(v[0] | static_cast<uint32_t>(v[1]) << 16, v[2] | static_cast<uint32_t>(v[3]) << 16);
  }
}

}  // namespace

// T from the partials, where a tiled product follows.
__global__ __launch_bounds__(256) void k_mx4_sum(const float *__restrict__ P, int S, int64_t n, float scale,
                                                 uint16_t *__restrict__ T) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float t = 0.f;
#pragma unroll 4
  for (int s = 0; s < S; ++s) t += P[s * n + i];
  T[i] = f32_to_bf16(scale * t);
}

// kMB: tiles of 16 tokens.  kFused: X is bf16 and rounded here (kMB == 1).
// kWaves waves take the slabs in turn.
template <int kMB, bool kFused, int kWaves>
__global__ __launch_bounds__(kWaves * 64, 4) void k_mx4_small(const SmallArgs a) {
  __shared__ float red[kWaves][kMB][256];
  __shared__ __attribute__((aligned(16))) uint16_t sT[16 * kMB][136];   // T, 128 columns and a skew
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * kMainRows;
  const int slabs = (a.K + 255) / 256, blocks = a.K / 32;
  const int wrow = min(n0 + nl, a.N - 1);
  const uint8_t *wc = a.wc + static_cast<int64_t>(wrow) * slabs * 128 + 16 * g;
  const uint8_t *ws = a.ws + static_cast<int64_t>(wrow) * 8;
  typedef Pass<kMB, kFused> pass_t;

  f32x4_t acc[kMB];
#pragma unroll
  for (int m = 0; m < kMB; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto load = [&](pass_t &p, int slab) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) p.w[h] = *reinterpret_cast<const i32x4_t *>(wc + slab * 128 + 64 * h);
    p.wb = *reinterpret_cast<const uint2 *>(ws + static_cast<int64_t>(slab) * a.N * 8);
    if constexpr (kFused) {
      const uint16_t *x = a.X + static_cast<int64_t>(min(nl, a.M - 1)) * a.K;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 *q = reinterpret_cast<const uint4 *>(x + 32 * min(slab * 8 + 4 * h + g, blocks - 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = q[i];
          p.raw[h][4 * i] = v.x;
          p.raw[h][4 * i + 1] = v.y;
          p.raw[h][4 * i + 2] = v.z;
          p.raw[h][4 * i + 3] = v.w;
        }
      }
    } else {
#pragma unroll
      for (int m = 0; m < kMB; ++m) {
        const int row = min(16 * m + nl, a.M - 1);
        const uint8_t *c = a.xc + (static_cast<int64_t>(row) * slabs + slab) * 128 + 16 * g;
#pragma unroll
        for (int h = 0; h < 2; ++h) p.x[m][h] = *reinterpret_cast<const i32x4_t *>(c + 64 * h);
        p.xb[m] = *reinterpret_cast<const uint2 *>(a.xs + (static_cast<int64_t>(slab) * a.M + row) * 8);
      }
    }
  };
  auto multiply = [&](const pass_t &p, int slab) __attribute__((always_inline)) {
    if (slab >= slabs) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int sw = static_cast<int>((h ? p.wb.y : p.wb.x) >> (8 * g));
      if constexpr (kFused) {
        i32x4_t x;
        uint32_t byte = round_block(p.raw[h], x);
        if (slab * 8 + 4 * h + g >= blocks) {   // past the row: W's fill is zero there, and so is X's
          x = i32x4_t{0, 0, 0, 0};
          byte = 0;
        }
        acc[0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(p.w[h]), widen(x), acc[0], 4, 4, 0, sw, 0,
                                                                  static_cast<int>(byte));
      } else {
#pragma unroll
        for (int m = 0; m < kMB; ++m) {
          const int sx = static_cast<int>((h ? p.xb[m].y : p.xb[m].x) >> (8 * g));
          acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(p.w[h]), widen(p.x[m][h]), acc[m], 4, 4, 0, sw, 0,
                                                                    sx);
        }
      }
    }
  };
  pass_t p;
  load(p, min(wave, slabs - 1));     // a wave without slabs reads the last one and multiplies nothing
  if (!kFused && a.r > 0) put_T<kMB, kWaves * 64, 6>(a, sT);   // its loads come behind the first pass's
  multiply(p, wave);
  for (int slab = wave + kWaves; slab < slabs; slab += kWaves) {
    load(p, slab);
    multiply(p, slab);
  }
#pragma unroll
  for (int m = 0; m < kMB; ++m) *reinterpret_cast<f32x4_t *>(&red[wave][m][4 * lane]) = acc[m];
  __syncthreads();
  if (wave >= kMB) return;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += *reinterpret_cast<const f32x4_t *>(&red[w][wave][4 * lane]);
  for (int j = 0; j < a.r; j += 32) {
    const bf16x8_t b = load8(a.B + static_cast<int64_t>(wrow) * a.r, j + 8 * g, a.r, (a.r & 7) == 0);
    const bf16x8_t t = *reinterpret_cast<const bf16x8_t *>(&sT[16 * wave + nl][j + 8 * g]);
    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, t, sum, 0, 0, 0);
  }
  // lane l holds columns n0 + 4 (l / 16) + e of token l % 16
  const int m = 16 * wave + nl, n = n0 + 4 * g;
  if (m >= a.M) return;
  uint16_t *y = a.Y + static_cast<int64_t>(m) * a.N + n;
  if ((a.N & 3) == 0) {
    if (n < a.N) *reinterpret_cast<uint2 *>(y) = make_uint2(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.N) y[e] = f32_to_bf16(sum[e]);
  }
}

namespace {

template <int kMB>
hipError_t launch_waves(const SmallArgs &a, hipStream_t s) {
  const int grid = (a.N + kMainRows - 1) / kMainRows;
  // Up to two workgroups a CU: 16 waves (64 x 4096 x 11008: 20.7 us, with 8
  // waves 21.1; 1 x 4096 x 4096: 3.7 and 3.5).  More: 8, of which more share a CU
  // (1 x 11008 x 4096: 6.7 us, with 16 waves 9.1; 16 x 11008 x 4096: 11.5 and 12.6).
  if (grid <= 512)
    hipLaunchKernelGGL((k_mx4_small<kMB, false, 16>), dim3(grid), dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL((k_mx4_small<kMB, false, 8>), dim3(grid), dim3(512), 0, s, a);
  return hipGetLastError();
}

// Without a LoRA pair and with a workgroup a CU at most, the main kernel rounds
// X itself and is the only launch: 1 x 4096 x 4096 takes 4.6 us, against 3.0
// + 3.9 us in two.  More workgroups would each round all of X again (1 x 11008
// x 4096: 12 us against 4.3 + 6.7), and T needs a launch before it anyway.
bool fused_ok(const SmallArgs &a) {
  return a.r == 0 && a.M <= kFusedTokens && (a.N + kMainRows - 1) / kMainRows <= kFusedGrid;
}

template <bool kFused>
hipError_t launch_main(const SmallArgs &a, hipStream_t s) {
  if constexpr (kFused) {
    hipLaunchKernelGGL((k_mx4_small<1, true, 16>), dim3((a.N + kMainRows - 1) / kMainRows), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
  if (a.M <= 16) return launch_waves<1>(a, s);
  if (a.M <= 32) return launch_waves<2>(a, s);
  return launch_waves<4>(a, s);
}

// The partial sums of X A^T (r > 0) and Q(X), one launch.
hipError_t launch_prep(const SmallArgs &a, const Mx4View &Xq, hipStream_t s) {
  const int64_t downs = a.r > 0 ? static_cast<int64_t>(a.S) * ((a.r + 15) / 16) * ((a.M + 15) / 16) : 0;
  const int64_t blocks = static_cast<int64_t>(a.M) * mx4_slabs(a.K) * 8;
  const dim3 grid(static_cast<uint32_t>(downs + (blocks + kPrepWaves * 64 - 1) / (kPrepWaves * 64))), block(kPrepWaves * 64);
  hipLaunchKernelGGL(k_mx4_prep, grid, block, 0, s, a, static_cast<int>(downs), Xq.codes, Xq.scales);
  return hipGetLastError();
}

}  // namespace

bool mx4_small_ok(int64_t M) { return M <= kMx4SmallMax; }

bool mx4_small_launch_ok(int64_t N) { return (N + kMainRows - 1) / kMainRows <= kMaxThreads / 512; }   // 8 waves (launch_waves)

size_t mx4_small_ws_bytes(int64_t M, int64_t K, int r) {
  return static_cast<size_t>((K + kSlice - 1) / kSlice) * M * r * sizeof(float);
}

hipError_t launch_mx4_small_matmul(const Mx4View &X, const Mx4View &W, const uint16_t *T, const uint16_t *B, int r,
                                   uint16_t *Y, hipStream_t s) {
  SmallArgs a{};
  a.xc = X.codes;
  a.xs = X.scales;
  a.wc = W.codes;
  a.ws = W.scales;
  a.B = B;
  a.T = T;
  a.Y = Y;
  a.M = static_cast<int>(X.rows);
  a.N = static_cast<int>(W.rows);
  a.K = static_cast<int>(X.cols);
  a.r = r;
  return launch_main<false>(a, s);
}

hipError_t launch_mx4_prep(const uint16_t *X, const Mx4View &Xq, const uint16_t *A, int r, float scale, uint16_t *T,
                           float *P, hipStream_t s) {
  SmallArgs a{};
  a.X = X;
  a.A = A;
  a.P = P;
  a.Tout = T;
  a.M = static_cast<int>(Xq.rows);
  a.K = static_cast<int>(Xq.cols);
  a.r = r;
  a.slice = kSlice;
  a.S = (a.K + a.slice - 1) / a.slice;
  a.scale = scale;
  const hipError_t e = launch_prep(a, Xq, s);
  if (e != hipSuccess) return e;
  const int64_t n = static_cast<int64_t>(a.M) * r;
  hipLaunchKernelGGL(k_mx4_sum, dim3(static_cast<uint32_t>((n + 255) / 256)), dim3(256), 0, s, P, a.S, n, scale, T);
  return hipGetLastError();
}

hipError_t launch_mx4_small_linear(const uint16_t *X, const Mx4View &W, const uint16_t *A, const uint16_t *B, int r,
                                   float scale, uint16_t *Y, uint16_t *Tout, float *P, const Mx4View &Xq, hipStream_t s) {
  SmallArgs a{};
  a.X = X;
  a.xc = Xq.codes;
  a.xs = Xq.scales;
  a.wc = W.codes;
  a.ws = W.scales;
  a.A = A;
  a.B = B;
  a.P = P;
  a.Y = Y;
  a.Tout = Tout;
  a.M = static_cast<int>(Xq.rows);
  a.N = static_cast<int>(W.rows);
  a.K = static_cast<int>(W.cols);
  a.r = r;
  a.slice = kSlice;
  a.S = (a.K + a.slice - 1) / a.slice;
  a.scale = scale;
  const bool fused = fused_ok(a);
  if (!fused) {
    const hipError_t e = launch_prep(a, Xq, s);
    if (e != hipSuccess) return e;
  }
  return fused ? launch_main<true>(a, s) : launch_main<false>(a, s);
}

}  // namespace qlora
