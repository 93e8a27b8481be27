// The MX4 linear layer at few tokens (M <= 64):
//     Y [M, N] = Q(X) W^T + T B^T,   T = bf16(scale X A^T)
// The weight's bytes bound it, then the latency of a launch's few loads, so W
// goes from memory straight into registers, every wave issues the loads of a
// pass before the first product, and there are two launches at most.
//
// k_mx4_prep: partial sums P of X A^T, one workgroup per (slice of the
//   columns, 32 adapter rows, 32 or 16 tokens); its 16 waves split the slice
//   and are summed in LDS in wave order.  From 17 tokens on, further
//   workgroups of the same launch round X to MX4.
// k_mx4_small: one workgroup per 16 weight rows, its 8 waves take slabs of 256
//   columns in turn: v_mfma_scale_f32_16x16x128 with W as the left operand
//   (lane l: row l % 16, block l / 16 of 128 columns) and 16 tokens a product
//   as the right one.  Up to 16 tokens a lane rounds the block of X that it
//   supplies itself, 32 bf16 of one token: the block's maximum needs no other
//   lane, and no third launch is made.  The waves' sums meet in LDS in wave
//   order; T B^T is added there from the partials' sum.
#include <algorithm>

#include "common.h"
#include "launch.h"

namespace qlora {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

constexpr int kPrepWaves = 16;
constexpr int kPrepRows = 32;         // adapter rows of a workgroup
constexpr int kMainWaves = 8;
constexpr int kMainRows = 16;         // weight rows of a workgroup
constexpr int kFusedMax = 16;         // tokens up to which the main kernel rounds X itself

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

// kMT: token tiles of 16 of a workgroup.  Workgroups from `downs` on round X.
template <int kMT>
__global__ __launch_bounds__(kPrepWaves * 64) void k_mx4_prep(const SmallArgs a, int downs, uint8_t *xc, uint8_t *xs) {
  __shared__ float red[kPrepWaves][2 * kMT][256];
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
  const int jts = (a.r + kPrepRows - 1) / kPrepRows, mts = (a.M + 16 * kMT - 1) / (16 * kMT);
  const int jt = blockIdx.x % jts, mt = blockIdx.x / jts % mts, s = blockIdx.x / (jts * mts);
  const int nl = lane & 15, g = lane >> 4;
  const int per = a.slice / kPrepWaves;               // columns of a wave: 64 or 128
  const int k0 = s * a.slice + wave * per;
  f32x4_t acc[2][kMT];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int m = 0; m < kMT; ++m) acc[j][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint16_t *ar[2], *xr[kMT];
#pragma unroll
  for (int j = 0; j < 2; ++j) ar[j] = a.A + static_cast<int64_t>(min(kPrepRows * jt + 16 * j + nl, a.r - 1)) * a.K;
#pragma unroll
  for (int m = 0; m < kMT; ++m) xr[m] = a.X + static_cast<int64_t>(min(16 * (kMT * mt + m) + nl, a.M - 1)) * a.K;
  for (int k = k0; k < min(k0 + per, a.K); k += 64) {   // K % 32 == 0: a 32-wide step is whole or absent
    bf16x8_t av[2][2], xv[2][kMT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = min(k + 32 * h, a.K - 32) + 8 * g;
#pragma unroll
      for (int j = 0; j < 2; ++j) av[h][j] = *reinterpret_cast<const bf16x8_t *>(ar[j] + c);
#pragma unroll
      for (int m = 0; m < kMT; ++m) xv[h][m] = *reinterpret_cast<const bf16x8_t *>(xr[m] + c);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (k + 32 * h < a.K) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int m = 0; m < kMT; ++m)
            acc[j][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[h][j], xv[h][m], acc[j][m], 0, 0, 0);
      }
  }
  // lane l holds adapter rows 4 (l / 16) + e of token l % 16
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int m = 0; m < kMT; ++m)
      *reinterpret_cast<f32x4_t *>(&red[wave][j * kMT + m][4 * lane]) = acc[j][m];
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kMT * 256; i += kPrepWaves * 64) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kPrepWaves; ++w) v += red[w][i >> 8][i & 255];
    const int l = (i & 255) >> 2, e = i & 3, t = i >> 8;
    const int j = kPrepRows * jt + 16 * (t / kMT) + 4 * (l >> 4) + e, m = 16 * (kMT * mt + t % kMT) + (l & 15);
    if (j < a.r && m < a.M) a.P[(static_cast<int64_t>(s) * a.M + m) * a.r + j] = v;
  }
}

// kMB: tiles of 16 tokens.  kFused: X is bf16 and rounded here (kMB == 1).
template <int kMB, bool kFused>
__global__ __launch_bounds__(kMainWaves * 64) void k_mx4_small(const SmallArgs a) {
  constexpr int kU = kMB > 2 ? 1 : 2;                // slabs of a pass
  __shared__ float red[kMainWaves][kMB][256];
  __shared__ __attribute__((aligned(16))) uint16_t sT[16 * kMB][136];   // T, 128 columns and a skew
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * kMainRows;
  const int slabs = (a.K + 255) / 256, blocks = a.K / 32;
  const int wrow = min(n0 + nl, a.N - 1);
  const uint8_t *wc = a.wc + static_cast<int64_t>(wrow) * slabs * 128 + 16 * g;
  const uint8_t *ws = a.ws + static_cast<int64_t>(wrow) * 8;

  f32x4_t acc[kMB];
#pragma unroll
  for (int m = 0; m < kMB; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int sl = wave * kU; sl < slabs; sl += kMainWaves * kU) {
    i32x4_t wv[kU][2], xv[kU][kMB][2];
    uint2 wb[kU], xb[kU][kMB];
    uint32_t raw[kFused ? kU : 1][2][16];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int slab = min(sl + u, slabs - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) wv[u][h] = *reinterpret_cast<const i32x4_t *>(wc + slab * 128 + 64 * h);
      wb[u] = *reinterpret_cast<const uint2 *>(ws + static_cast<int64_t>(slab) * a.N * 8);
      if constexpr (kFused) {
        const uint16_t *x = a.X + static_cast<int64_t>(min(nl, a.M - 1)) * a.K;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 *p = reinterpret_cast<const uint4 *>(x + 32 * min(slab * 8 + 4 * h + g, blocks - 1));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = p[i];
            raw[u][h][4 * i] = v.x;
            raw[u][h][4 * i + 1] = v.y;
            raw[u][h][4 * i + 2] = v.z;
            raw[u][h][4 * i + 3] = v.w;
          }
        }
      } else {
#pragma unroll
        for (int m = 0; m < kMB; ++m) {
          const int row = min(16 * m + nl, a.M - 1);
          const uint8_t *c = a.xc + (static_cast<int64_t>(row) * slabs + slab) * 128 + 16 * g;
#pragma unroll
          for (int h = 0; h < 2; ++h) xv[u][m][h] = *reinterpret_cast<const i32x4_t *>(c + 64 * h);
          xb[u][m] = *reinterpret_cast<const uint2 *>(a.xs + (static_cast<int64_t>(slab) * a.M + row) * 8);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (sl + u >= slabs) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sw = (h ? wb[u].y : wb[u].x) >> (8 * g);
        if constexpr (kFused) {
          uint32_t byte = round_block(raw[u][h], xv[u][0][h]);
          if ((sl + u) * 8 + 4 * h + g >= blocks) {   // past the row: W's fill is zero there, and so is X's
            xv[u][0][h] = i32x4_t{0, 0, 0, 0};
            byte = 0;
          }
          acc[0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(wv[u][h]), widen(xv[u][0][h]), acc[0], 4, 4, 0,
                                                                    static_cast<int>(sw), 0, static_cast<int>(byte));
        } else {
#pragma unroll
          for (int m = 0; m < kMB; ++m) {
            const uint32_t sx = (h ? xb[u][m].y : xb[u][m].x) >> (8 * g);
            acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(wv[u][h]), widen(xv[u][m][h]), acc[m], 4, 4, 0,
                                                                      static_cast<int>(sw), 0, static_cast<int>(sx));
          }
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kMB; ++m) *reinterpret_cast<f32x4_t *>(&red[wave][m][4 * lane]) = acc[m];

  if (a.r > 0) {
    // T [M, r] into LDS, zero up to the next 32 columns
    const int rp = (a.r + 31) / 32 * 32;
    for (int i = threadIdx.x; i < 16 * kMB * rp; i += kMainWaves * 64) {
      const int m = i / rp, j = i - m * rp;
      uint16_t v = 0;
      if (m < a.M && j < a.r) {
        if (a.T) {
          v = a.T[static_cast<int64_t>(m) * a.r + j];
        } else {
          float t = 0.f;
          for (int s = 0; s < a.S; ++s) t += a.P[(static_cast<int64_t>(s) * a.M + m) * a.r + j];
          v = f32_to_bf16(a.scale * t);
          if (blockIdx.x == 0 && a.Tout) a.Tout[static_cast<int64_t>(m) * a.r + j] = v;
        }
      }
      sT[m][j] = v;
    }
  }
  __syncthreads();
  if (wave >= kMB) return;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kMainWaves; ++w) sum += *reinterpret_cast<const f32x4_t *>(&red[w][wave][4 * lane]);
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

int slice_of(int M) { return M <= kFusedMax ? 1024 : 2048; }

template <bool kFused>
hipError_t launch_main(const SmallArgs &a, hipStream_t s) {
  const dim3 grid((a.N + kMainRows - 1) / kMainRows), block(kMainWaves * 64);
  if constexpr (kFused) {
    hipLaunchKernelGGL((k_mx4_small<1, true>), grid, block, 0, s, a);
  } else if (a.M <= 16) {
    hipLaunchKernelGGL((k_mx4_small<1, false>), grid, block, 0, s, a);
  } else if (a.M <= 32) {
    hipLaunchKernelGGL((k_mx4_small<2, false>), grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL((k_mx4_small<4, false>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

bool mx4_small_ok(int64_t M) { return M <= kMx4SmallMax; }

size_t mx4_small_ws_bytes(int64_t M, int64_t K, int r) {
  const int64_t S = (K + slice_of(static_cast<int>(M)) - 1) / slice_of(static_cast<int>(M));
  return static_cast<size_t>(S) * M * r * sizeof(float);
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
  a.slice = slice_of(a.M);
  a.S = (a.K + a.slice - 1) / a.slice;
  a.scale = scale;
  const bool fused = a.M <= kFusedMax;
  const int mt = fused ? 1 : 2;
  const int downs = r > 0 ? a.S * ((r + kPrepRows - 1) / kPrepRows) * ((a.M + 16 * mt - 1) / (16 * mt)) : 0;
  const int64_t blocks = fused ? 0 : static_cast<int64_t>(a.M) * mx4_slabs(a.K) * 8;
  const int64_t rounds = (blocks + kPrepWaves * 64 - 1) / (kPrepWaves * 64);
  const dim3 grid(static_cast<uint32_t>(downs + rounds)), block(kPrepWaves * 64);
  if (grid.x > 0) {
    if (fused)
      hipLaunchKernelGGL(k_mx4_prep<1>, grid, block, 0, s, a, downs, Xq.codes, Xq.scales);
    else
      hipLaunchKernelGGL(k_mx4_prep<2>, grid, block, 0, s, a, downs, Xq.codes, Xq.scales);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return fused ? launch_main<true>(a, s) : launch_main<false>(a, s);
}

}  // namespace qlora
