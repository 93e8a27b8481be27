// Products of two MX4 arrays on gfx950's scaled matrix instructions:
//     Y [M, N] = X W^T + T B^T        X [M, K], W [N, K] in MX4; T, B bf16
// sum over blocks b of 2^(sx + sw) sum_k x_k w_k: v_mfma_scale_f32_32x32x64
// takes the codes and both block scales, so nothing is expanded.  Products of
// two E2M1 values are exact; sums are fp32.
//
//  * 64 kFM x 128 kFN output tile, 8 waves as 2 x 4, each 32 kFM x 32 kFN of
//    fp32 accumulators; contraction step 256 (a slab: 128 bytes of codes a
//    row, 8 scale bytes).
//  * Codes and scales go global -> LDS by DMA one step ahead (two stages).
//    A 16-byte chunk of a row is one block of 32 codes, and lane l of the
//    instruction takes row l % 32 and block l / 32 of a 64-wide sub-step, so
//    the operand reads are those of a bf16 tile with 64 columns: chunks
//    XOR-swizzled by row, no bank conflicts.
//  * Scales: 8 bytes a row and step.  A lane shifts its row's words by 8 (l /
//    32) bits; bytes 0 and 2 of the first word are then its blocks' scales in
//    sub-steps 0 and 1, of the second in 2 and 3, picked by the instruction.
//  * The LoRA term is one (r <= 64) or two more steps on bf16 MFMA into the
//    same accumulators.
#include "common.h"
#include "launch.h"
#include "lds_dma.h"
#include "tile.h"

namespace qlora {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kMxMmThreads = 512;
constexpr int kMxBand = 4;   // tile rows of a band (see tile_of)

struct Mx4Args {
  const uint8_t *xc, *xs, *wc, *ws;
  const uint16_t *T, *B;
  uint16_t *Y;
  int M, N, r;
  int KT;            // slabs
  int trows, tcols;
};

// 4 bytes a lane, global -> LDS (see dma16).
__device__ __forceinline__ void dma4(const void *src, uint32_t dst) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "{m0}"(dst) : "memory");
}

// Consecutive workgroups go to the 8 XCDs in turn; consecutive tiles are
// given to one XCD, in bands of kMxBand tile rows, column by column, so that
// the tiles an XCD runs together share rows of X and of W in its L2.
__device__ __forceinline__ void tile_of(const Mx4Args &a, int &tr, int &tc) {
  int id = blockIdx.x;
  const int nt = gridDim.x;
  if ((nt & 7) == 0) id = (blockIdx.x & 7) * (nt >> 3) + (blockIdx.x >> 3);
  const int band = id / (kMxBand * a.tcols);
  const int h = min(kMxBand, a.trows - band * kMxBand);
  const int j = id - band * kMxBand * a.tcols;
  tc = j / h;
  tr = band * kMxBand + j % h;
}

// Codes of rows row0 .. row0 + kRows - 1 (past the last: that row again, its
// results are not stored) of one slab into a swizzled stage.
template <int kRows>
__device__ __forceinline__ void dma_codes(uint8_t *stage, const uint8_t *codes, int64_t pitch, int row0, int rows, int kt,
                                          int wave, int lane) {
#pragma unroll
  for (int j = 0; j < kRows / 64; ++j) {
    const int u = wave * (kRows / 64) + j;
    const int row = u * 8 + (lane >> 3);
    const int chunk = (lane & 7) ^ ((row & 7) ^ ((row >> 3) & 1));
    const uint32_t dst = __builtin_amdgcn_readfirstlane(lds_addr(stage) + u * 1024);
    dma16(codes + static_cast<int64_t>(min(row0 + row, rows - 1)) * pitch + kt * 128 + chunk * 16, dst);
  }
}

// Their scales: 8 bytes a row, 32 rows a wave instruction.
__device__ __forceinline__ void dma_scales(uint8_t *stage, const uint8_t *scales, int row0, int rows, int kt, int u,
                                           int lane) {
  const int row = min(row0 + 32 * u + (lane >> 1), rows - 1);
  const uint32_t dst = __builtin_amdgcn_readfirstlane(lds_addr(stage) + u * 256);
  dma4(scales + (static_cast<int64_t>(kt) * rows + row) * 8 + 4 * (lane & 1), dst);
}

__device__ __forceinline__ i32x8_t widen(i32x4_t v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }

// One 32 x 32 x 64 product; s: sub-step (its scale byte), sa, sb: the words.
template <int kByte>
__device__ __forceinline__ f32x16_t mfma4(i32x4_t a, i32x4_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), widen(b), c, 4, 4, kByte, static_cast<int>(sa), kByte,
                                                         static_cast<int>(sb));
}

template <int kFM, int kFN>
struct Scales {
  uint2 a[kFM], b[kFN];
};

// Narrow bf16 [rows, r] (T or B), columns j0 .. j0 + 63, into a 128-byte-row
// stage of kRows rows; zero past r and past `rows`.
template <int kRows>
__device__ __forceinline__ void stage_narrow(uint8_t *stage, const uint16_t *src, int r, int row0, int rows, int j0) {
  const bool vec = (r & 7) == 0;
  for (int idx = threadIdx.x; idx < kRows * 8; idx += kMxMmThreads) {
    const int row = idx >> 3, c = idx & 7;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row0 + row < rows) {
      const uint16_t *p = src + static_cast<int64_t>(row0 + row) * r + j0 + 8 * c;
      if (vec) {
        if (j0 + 8 * c < r) v = *reinterpret_cast<const uint4 *>(p);
      } else {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = j0 + 8 * c + e < r ? p[e] : 0u;
        v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      }
    }
    *reinterpret_cast<uint4 *>(stage + swz128(row, c)) = v;
  }
}

}  // namespace

template <int kFM, int kFN>
__global__ __launch_bounds__(kMxMmThreads) void k_mx4_matmul(const Mx4Args args) {
  constexpr int kBM = 64 * kFM, kBN = 128 * kFN;
  __shared__ __attribute__((aligned(16))) uint8_t sX[2][kBM * 128];
  __shared__ __attribute__((aligned(16))) uint8_t sW[2][kBN * 128];
  __shared__ __attribute__((aligned(16))) uint8_t sSx[2][kBM * 8];
  __shared__ __attribute__((aligned(16))) uint8_t sSw[2][kBN * 8];

  int tr, tc;
  tile_of(args, tr, tc);
  const int M = args.M, N = args.N, r = args.r, KT = args.KT;
  const int64_t pitch = static_cast<int64_t>(KT) * 128;
  const int m0 = tr * kBM, n0 = tc * kBN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int lr = lane & 31, lh = lane >> 5;

  auto dma = [&](int st, int kt) __attribute__((always_inline)) {
    dma_codes<kBM>(sX[st], args.xc, pitch, m0, M, kt, wave, lane);
    dma_codes<kBN>(sW[st], args.wc, pitch, n0, N, kt, wave, lane);
#pragma unroll
    for (int u = wave; u < (kBM + kBN) / 32; u += 8) {
      if (u < kBM / 32)
        dma_scales(sSx[st], args.xs, m0, M, kt, u, lane);
      else
        dma_scales(sSw[st], args.ws, n0, N, kt, u - kBM / 32, lane);
    }
  };
  uint32_t xo[4], wo[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    xo[s] = static_cast<uint32_t>(swz128(32 * kFM * wm + lr, 2 * s + lh));
    wo[s] = static_cast<uint32_t>(swz128(32 * kFN * wn + lr, 2 * s + lh));
  }
  f32x16_t acc[kFM][kFN];
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  dma(0, 0);
  raw_barrier<wait_imm(0, 0)>();
  for (int kt = 0; kt < KT; ++kt) {
    const int st = kt & 1;
    if (kt + 1 < KT) dma(st ^ 1, kt + 1);
    Scales<kFM, kFN> sc;
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
      const uint2 v = *reinterpret_cast<const uint2 *>(sSx[st] + (32 * kFM * wm + 32 * i + lr) * 8);
      sc.a[i] = make_uint2(v.x >> (8 * lh), v.y >> (8 * lh));
    }
#pragma unroll
    for (int j = 0; j < kFN; ++j) {
      const uint2 v = *reinterpret_cast<const uint2 *>(sSw[st] + (32 * kFN * wn + 32 * j + lr) * 8);
      sc.b[j] = make_uint2(v.x >> (8 * lh), v.y >> (8 * lh));
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      i32x4_t a[kFM], b[kFN];
#pragma unroll
      for (int i = 0; i < kFM; ++i) a[i] = *reinterpret_cast<const i32x4_t *>(sX[st] + xo[s] + 4096 * i);
#pragma unroll
      for (int j = 0; j < kFN; ++j) b[j] = *reinterpret_cast<const i32x4_t *>(sW[st] + wo[s] + 4096 * j);
#pragma unroll
      for (int i = 0; i < kFM; ++i)
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          const uint32_t sa = s < 2 ? sc.a[i].x : sc.a[i].y, sb = s < 2 ? sc.b[j].x : sc.b[j].y;
          acc[i][j] = (s & 1) ? mfma4<2>(a[i], b[j], acc[i][j], sa, sb) : mfma4<0>(a[i], b[j], acc[i][j], sa, sb);
        }
    }
    raw_barrier<wait_imm(0, 0)>();
  }
  for (int j0 = 0; j0 < r; j0 += 64) {
    stage_narrow<kBM>(sX[0], args.T, r, m0, M, j0);
    stage_narrow<kBN>(sW[0], args.B, r, n0, N, j0);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < kFM; ++i)
#pragma unroll
        for (int j = 0; j < kFN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              *reinterpret_cast<const bf16x8_t *>(sX[0] + xo[s] + 4096 * i),
              *reinterpret_cast<const bf16x8_t *>(sW[0] + wo[s] + 4096 * j), acc[i][j], 0, 0, 0);
    __syncthreads();
  }

  // Epilogue: the wave's block as bf16 through its own part of the stages (no
  // wave reads them any more), 16 bytes a lane to memory.  Accumulator layout:
  // lane l holds column l % 32, element e row 8 (e / 4) + 4 (l / 32) + e % 4.
  constexpr int kRowBytes = 64 * kFN;                  // the wave's 32 kFN columns
  constexpr int kChunks = kRowBytes / 16;
  uint8_t *region = &sX[0][0] + wave * (32 * kFM * kRowBytes);
  static_assert(8 * 32 * kFM * kRowBytes <= 2 * kBM * 128 || kFM * kFN == 8, "");
  if constexpr (kFM * kFN == 8) region = (wave < 4 ? &sX[0][0] : &sW[0][0]) + (wave & 3) * (32 * kFM * kRowBytes);
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int rr = 32 * i + 8 * (e >> 2) + 4 * lh + (e & 3);
        const int cc = 32 * j + lr;
        *reinterpret_cast<uint16_t *>(region + rr * kRowBytes + 16 * ((cc >> 3) ^ (rr & (kChunks - 1))) + 2 * (cc & 7)) =
            f32_to_bf16(acc[i][j][e]);
      }
  __builtin_amdgcn_s_waitcnt(wait_imm(63, 0));
  const bool vec = (N & 7) == 0;
#pragma unroll 4
  for (int t = 0; t < 32 * kFM * kChunks / 64; ++t) {
    const int idx = t * 64 + lane;
    const int rr = idx / kChunks, c = idx % kChunks;
    const uint4 v = *reinterpret_cast<const uint4 *>(region + rr * kRowBytes + 16 * (c ^ (rr & (kChunks - 1))));
    const int gr = m0 + 32 * kFM * wm + rr, gc = n0 + 32 * kFN * wn + 8 * c;
    if (gr >= M) continue;
    uint16_t *p = args.Y + static_cast<int64_t>(gr) * N + gc;
    if (vec) {
      if (gc < N) *reinterpret_cast<uint4 *>(p) = v;
    } else {
      const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (gc + e < N) p[e] = static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1)));
    }
  }
}

namespace {

template <int kFM, int kFN>
hipError_t launch_tiles(Mx4Args a, hipStream_t s) {
  a.trows = (a.M + 64 * kFM - 1) / (64 * kFM);
  a.tcols = (a.N + 128 * kFN - 1) / (128 * kFN);
  hipLaunchKernelGGL((k_mx4_matmul<kFM, kFN>), dim3(static_cast<uint32_t>(a.trows) * a.tcols), dim3(kMxMmThreads), 0, s,
                     a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_matmul(const Mx4View &X, const Mx4View &W, const uint16_t *T, const uint16_t *B, int r, uint16_t *Y,
                             hipStream_t s) {
  Mx4Args a{};
  a.xc = X.codes;
  a.xs = X.scales;
  a.wc = W.codes;
  a.ws = W.scales;
  a.T = T;
  a.B = B;
  a.Y = Y;
  a.M = static_cast<int>(X.rows);
  a.N = static_cast<int>(W.rows);
  a.r = r;
  a.KT = static_cast<int>(mx4_slabs(X.cols));
  // The small tile where the large one leaves compute units without work.
  const int64_t large = ((X.rows + 255) / 256) * ((W.rows + 255) / 256);
  return large >= 256 ? launch_tiles<4, 2>(a, s) : launch_tiles<2, 1>(a, s);
}

}  // namespace qlora
