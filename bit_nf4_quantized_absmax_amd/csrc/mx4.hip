// MX4 codec: arrays [rows, cols] in microscaled 4-bit floating point.
//
// A block of 32 consecutive elements of a row shares the scale 2^s and holds
// E2M1 codes (sign, then the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6):
//     s = max(floor(log2(max |x|)) - 2, -127),   byte = s + 127
//     code = x / 2^s to the nearest level, ties to the even code, clipped to 6
// so that the block's largest element lands in [4, 8).  With the exponent
// field E of fp32 max |x| (0 for zero and subnormals) the byte is max(E - 2,
// 0): no logarithm.  A block that holds a NaN or an infinity gets the byte 255
// and zero codes; every element of it decodes to NaN.
//
// Layout: rows are filled up to Kp, the next multiple of 256, with zero codes
// and zero bytes.
//   codes  [rows][Kp / 2]         element 2 j in the low half of byte j
//   scales [Kp / 256][rows][8]    the 8 blocks of a 256-wide slab of a row
// A slab's scales lie together for neighbouring rows, so the product's tiles
// read them as one run; its codes are 128 bytes a row, a whole cache line.
//
// Both directions move bytes and nothing else counts: 2.53 to 4.53 bytes an
// element.  A group of 32 lanes holds one slab of one row, 8 elements a lane
// (16-byte loads of 16-bit types); four lanes share a block, whose maximum
// goes over them in two DPP steps.
#include "common.h"
#include "launch.h"
#include "tile.h"

namespace qlora {

namespace {

constexpr int kMxThreads = 256;                  // 8 groups of 32 lanes
constexpr int kMxGroups = kMxThreads / 32;
constexpr int kDeRows = 2;                       // rows a lane decodes

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xF, 0xF, true));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kRowRor4 = 0x124, kRowRor8 = 0x128;

// 8 elements of a row as fp32.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __bf16 *p, float (&x)[8]) {
  const bf16x8_t v = *reinterpret_cast<const bf16x8_t *>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(v[i]);
}
__device__ __forceinline__ void load8(const _Float16 *p, float (&x)[8]) {
  typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
  const f16x8_t v = *reinterpret_cast<const f16x8_t *>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(v[i]);
}

}  // namespace

// One workgroup: 8 rows of one slab.  A load a lane in flight is enough with
// 8 workgroups a CU: 22016 x 8192 takes 99.8 us from bf16 and 158 from fp32 (4.6
// and 5.2 TB/s), with four rows a lane 108 and 160; 16 x 4096 2.3 and 2.8.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void k_mx4_quantize(const T *__restrict__ X, int64_t rows, int64_t cols,
                                                             int64_t slabs, uint8_t *__restrict__ codes,
                                                             uint8_t *__restrict__ scales) {
  const int64_t slab = blockIdx.x % slabs;
  const int64_t row = static_cast<int64_t>(blockIdx.x / slabs) * kMxGroups + (threadIdx.x >> 5);
  if (row >= rows) return;   // whole groups of 32 lanes
  const int l = threadIdx.x & 31;
  const int64_t c = slab * 256 + 8 * l;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < cols) load8(X + row * cols + c, x);
  uint32_t top = 0;   // largest |x| as bits: an infinity or a NaN compares above every number
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  top = max(top, dpp<kQuadXor1>(top));
  top = max(top, dpp<kQuadXor2>(top));
  const uint32_t e = top >> 23;
  const uint32_t byte = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
  uint32_t code = 0;
  if (byte != 255u) {
    const float f = mx4_scale(byte);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[0], x[1], f, 0);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[2], x[3], f, 1);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[4], x[5], f, 2);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[6], x[7], f, 3);
  }
  // the bytes of four blocks into one word (16 lanes)
  uint32_t word = byte << (8 * ((l >> 2) & 3));
  word |= dpp<kRowRor4>(word);
  word |= dpp<kRowRor8>(word);
  *reinterpret_cast<uint32_t *>(codes + row * (slabs * 128) + slab * 128 + 4 * l) = code;
  if ((l & 15) == 0) *reinterpret_cast<uint32_t *>(scales + (slab * rows + row) * 8 + (l >> 4) * 4) = word;
}

// The values, exact in bf16: a level has two significant bits, and 2^s times
// 0.5 reaches 2^-128, a bf16 subnormal.  Two rows a lane: 22016 x 8192 takes 67
// us (6.8 TB/s, most of it stores), with one 85, with four 74.
__global__ __launch_bounds__(kMxThreads) void k_mx4_dequantize(const uint8_t *__restrict__ codes,
                                                               const uint8_t *__restrict__ scales, int64_t rows,
                                                               int64_t cols, int64_t slabs, uint16_t *__restrict__ out) {
  const int64_t slab = blockIdx.x % slabs;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / slabs) * (kMxGroups * kDeRows) + (threadIdx.x >> 5);
  const int l = threadIdx.x & 31;
  const int64_t c = slab * 256 + 8 * l;
  if (c >= cols) return;
  constexpr int kU = kDeRows;
  uint32_t code[kU], byte[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t row = min(row0 + kMxGroups * u, rows - 1);
    code[u] = *reinterpret_cast<const uint32_t *>(codes + row * (slabs * 128) + slab * 128 + 4 * l);
    byte[u] = scales[(slab * rows + row) * 8 + (l >> 2)];
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t row = row0 + kMxGroups * u;
    const float f = mx4_scale(byte[u]);
    uint32_t v[4];
    v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[u], f, 0));
    v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[u], f, 1));
    v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[u], f, 2));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[u], f, 3));
    if (byte[u] == 255u) v[0] = v[1] = v[2] = v[3] = 0x7FC07FC0u;
    if (row < rows) *reinterpret_cast<uint4 *>(out + row * cols + c) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// 64 x 64 values of W transposed by way of LDS, or (workgroups from `tiles` on) up
// to 64 rows by 64 columns of A.  4096 x 4096: 14.6 us (2.9 TB/s), in rows 8.1: whole
// cache lines are stored, but a quarter of one is read at a time.
__global__ __launch_bounds__(kMxThreads) void k_mx4_transpose(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, int64_t N, int64_t K,
                                                              const uint16_t *__restrict__ A, int r, int64_t tiles,
                                                              uint16_t *__restrict__ Wt, uint16_t *__restrict__ At) {
  __shared__ __attribute__((aligned(16))) uint16_t sh[64][72];   // [column][row] and a skew
  const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
  const int64_t cols = K / 64, slabs = (K + 255) / 256;
  if (blockIdx.x < tiles) {
    const int64_t n = blockIdx.x / cols * 64, k = blockIdx.x % cols * 64;
    const uint2 c = *reinterpret_cast<const uint2 *>(codes + (n + row) * (slabs * 128) + k / 2 + 8 * part);
    const int64_t block = k / 32 + (part >> 1);
    const uint32_t byte = scales[(block / 8 * N + n + row) * 8 + block % 8];
    const float f = mx4_scale(byte);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t code = h ? c.y : c.x;
      uint32_t v[4];
      v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, f, 0));
      v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, f, 1));
      v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, f, 2));
      v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, f, 3));
      if (byte == 255u) v[0] = v[1] = v[2] = v[3] = 0x7FC07FC0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) sh[16 * part + 8 * h + e][row] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
    }
    __syncthreads();
    uint4 *out = reinterpret_cast<uint4 *>(Wt + (k + row) * N + n + 16 * part);
    out[0] = *reinterpret_cast<const uint4 *>(&sh[row][16 * part]);
    out[1] = *reinterpret_cast<const uint4 *>(&sh[row][16 * part + 8]);
    return;
  }
  const int64_t at = blockIdx.x - tiles, k = at % cols * 64;
  const int j0 = static_cast<int>(at / cols) * 64;
  if (j0 + row < r) {
    const uint16_t *a = A + static_cast<int64_t>(j0 + row) * K + k + 16 * part;
#pragma unroll
    for (int e = 0; e < 16; ++e) sh[16 * part + e][row] = a[e];
  }
  __syncthreads();
  for (int e = 0; e < 16; ++e)
    if (j0 + 16 * part + e < r) At[(k + row) * r + j0 + 16 * part + e] = sh[row][16 * part + e];
}

namespace {

// Workgroups of `each` rows of a slab.
int64_t mx4_groups(int64_t rows, int64_t cols, int each) { return (rows + each - 1) / each * mx4_slabs(cols); }

dim3 mx4_grid(const Mx4View &a, int each) { return dim3(static_cast<uint32_t>(mx4_groups(a.rows, a.cols, each))); }

template <typename T>
hipError_t quantize_as(const T *X, const Mx4View &a, hipStream_t s) {
  hipLaunchKernelGGL(k_mx4_quantize<T>, mx4_grid(a, kMxGroups), dim3(kMxThreads), 0, s, X, a.rows, a.cols,
                     mx4_slabs(a.cols), a.codes, a.scales);
  return hipGetLastError();
}

}  // namespace

bool mx4_quantize_ok(int64_t rows, int64_t cols) { return mx4_groups(rows, cols, kMxGroups) <= kMaxThreads / kMxThreads; }

bool mx4_dequantize_ok(int64_t rows, int64_t cols) {
  return mx4_groups(rows, cols, kMxGroups * kDeRows) <= kMaxThreads / kMxThreads;
}

hipError_t launch_mx4_quantize(const void *X, int in_type, const Mx4View &a, hipStream_t s) {
  if (in_type == 0) return quantize_as(static_cast<const float *>(X), a, s);
  if (in_type == 1) return quantize_as(static_cast<const __bf16 *>(X), a, s);
  return quantize_as(static_cast<const _Float16 *>(X), a, s);
}

hipError_t launch_mx4_dequantize(const Mx4View &a, uint16_t *out, hipStream_t s) {
  hipLaunchKernelGGL(k_mx4_dequantize, mx4_grid(a, kMxGroups * kDeRows), dim3(kMxThreads), 0, s, a.codes, a.scales, a.rows,
                     a.cols, mx4_slabs(a.cols), out);
  return hipGetLastError();
}

hipError_t launch_mx4_transpose(const Mx4View &W, const uint16_t *A, int r, uint16_t *Wt, uint16_t *At, hipStream_t s) {
  const int64_t tiles = W.rows / 64 * (W.cols / 64);
  hipLaunchKernelGGL(k_mx4_transpose, dim3(static_cast<uint32_t>(tiles + W.cols / 64 * ((r + 63) / 64))), dim3(kMxThreads), 0, s,
                     W.codes, W.scales, W.rows, W.cols, A, r, tiles, Wt, At);
  return hipGetLastError();
}

}  // namespace qlora
