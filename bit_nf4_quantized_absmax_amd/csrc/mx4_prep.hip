// X of the MX4 linear layer in one pass, for many tokens and an adapter of up to
// 16 rows: rounded to MX4 and multiplied by the adapter,
//     Q(X)    and    T [M, r] = bf16(scale X A^T),
// so that X's bytes, which bound both, are read once.
//
// One workgroup per 32 tokens; its 16 waves take slabs of 256 columns in turn.
// The bf16 MFMA 16x16x32 wants lane l to hold 8 columns (8 (l / 16) ..) of row
// l % 16, so a block of 32 columns lies across the four quarters of a wave.
// Over four blocks (128 columns) three 4 x 4 transposes between quarters, each
// four half- and quarter-wave swaps, bring the partial maxima of block g to
// quarter g, its scale back to all, and its 16 bytes of codes to quarter g,
// which stores them whole.  A comes from the L2.  The waves' products meet in
// LDS, the upper eight's first, and are summed in wave order.
//
// 8192 x 4096, r = 8: 23 us, 3.6 TB/s of X's bytes and the codes' (LoRA product and
// codec, two launches: 31; 8192 x 11008: 65 and 82).  Bound by the chain of a
// workgroup's steps, one workgroup a compute unit: 64 adapter rows, four times
// A's loads and products in that chain, take 37 us against 34 in two launches, and
// 27 against 19 for 4096 tokens, so they are not made here.
#include "common.h"
#include "launch.h"
#include "tile.h"

namespace qlora {

namespace {

constexpr int kRowsWaves = 16;
constexpr int kRowsTokens = 32;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// d[s] of quarter g becomes d[g] of quarter s.
__device__ __forceinline__ void transpose4(uint32_t (&d)[4]) {
  const u32x2_t a = __builtin_amdgcn_permlane16_swap(d[0], d[1], false, false);
  const u32x2_t b = __builtin_amdgcn_permlane16_swap(d[2], d[3], false, false);
  const u32x2_t c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const u32x2_t e = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  d[0] = c[0];
  d[1] = e[0];
  d[2] = c[1];
  d[3] = e[1];
}

// Largest |x| of 8 bf16, as bits.
__device__ __forceinline__ uint32_t top_of(const uint4 &v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  u16x2_t t = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2_t, w[i] & 0x7FFF7FFFu));
  return max(static_cast<uint32_t>(t[0]), static_cast<uint32_t>(t[1]));
}

}  // namespace

__global__ __launch_bounds__(kRowsWaves * 64) void k_mx4_rows(const uint16_t *__restrict__ X, int M, int K,
                                                              const uint16_t *__restrict__ A, int r, float scale,
                                                              uint16_t *__restrict__ T, uint8_t *__restrict__ codes,
                                                              uint8_t *__restrict__ scales) {
  __shared__ float red[kRowsWaves / 2][2][256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, g = lane >> 4;
  const int m0 = blockIdx.x * kRowsTokens;
  const int slabs = (K + 255) / 256;
  const uint16_t *xr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) xr[i] = X + static_cast<int64_t>(min(m0 + 16 * i + nl, M - 1)) * K + 8 * g;

  f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  for (int half = 2 * wave; half < 2 * slabs; half = (half & 1) ? half + 2 * kRowsWaves - 1 : half + 1) {
    const int k0 = half * 128;
    uint4 x[2][4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i][s] = *reinterpret_cast<const uint4 *>(xr[i] + min(k0 + 32 * s, K - 32));
        if (k0 + 32 * s >= K) x[i][s] = make_uint4(0, 0, 0, 0);   // K % 32 == 0: a block is whole or absent
      }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const bf16x8_t a =
          *reinterpret_cast<const bf16x8_t *>(A + static_cast<int64_t>(min(nl, r - 1)) * K + min(k0 + 32 * s, K - 32) + 8 * g);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, x[i][s]), acc[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t top[4], f[4], code[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) top[s] = top_of(x[i][s]);
      transpose4(top);                                     // quarter g: block g's four maxima
      const uint32_t e = max(max(top[0], top[1]), max(top[2], top[3])) >> 7;
      const uint32_t byte = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
#pragma unroll
      for (int s = 0; s < 4; ++s) f[s] = byte;
      transpose4(f);                                       // every quarter: the bytes of blocks 0 .. 3
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float q = mx4_scale(f[s]);
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x[i][s].x), q, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x[i][s].y), q, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x[i][s].z), q, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, x[i][s].w), q, 3);
        code[s] = f[s] == 255u ? 0u : c;
      }
      transpose4(code);                                    // quarter g: block g's 16 bytes
      const int m = m0 + 16 * i + nl;
      if (m < M) {
        *reinterpret_cast<uint4 *>(codes + static_cast<int64_t>(m) * slabs * 128 + half * 64 + 16 * g) =
            make_uint4(code[0], code[1], code[2], code[3]);
        if (g == 0)
          *reinterpret_cast<uint32_t *>(scales + (static_cast<int64_t>(half >> 1) * M + m) * 8 + 4 * (half & 1)) =
              f[0] | f[1] << 8 | f[2] << 16 | f[3] << 24;
      }
    }
  }
  // lane l holds adapter rows 4 (l / 16) + e of token l % 16
  constexpr int kHalf = kRowsWaves / 2;
  if (wave >= kHalf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<f32x4_t *>(&red[wave - kHalf][i][4 * lane]) = acc[i];
  }
  __syncthreads();
  if (wave < kHalf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f32x4_t *p = reinterpret_cast<f32x4_t *>(&red[wave][i][4 * lane]);
      *p = acc[i] + *p;
    }
  }
  __syncthreads();
  const int q = threadIdx.x;
  if (q >= 2 * 256) return;
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kHalf; ++w) v += red[w][q >> 8][q & 255];
  const int l = (q & 255) >> 2;
  const int j = 4 * (l >> 4) + (q & 3), m = m0 + 16 * (q >> 8) + (l & 15);
  if (j < r && m < M) T[static_cast<int64_t>(m) * r + j] = f32_to_bf16(scale * v);
}

hipError_t launch_mx4_rows(const uint16_t *X, const Mx4View &Xq, const uint16_t *A, int r, float scale, uint16_t *T,
                           hipStream_t s) {
  const int M = static_cast<int>(Xq.rows), K = static_cast<int>(Xq.cols);
  hipLaunchKernelGGL(k_mx4_rows, dim3((M + kRowsTokens - 1) / kRowsTokens), dim3(kRowsWaves * 64), 0, s, X, M, K, A, r, scale,
                     T, Xq.codes, Xq.scales);
  return hipGetLastError();
}

}  // namespace qlora
