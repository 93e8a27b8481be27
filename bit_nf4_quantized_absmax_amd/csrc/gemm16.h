// The bf16 product of two matrices on gfx950's matrix instructions, as a device
// function whose callers add what follows it (a row's softmax, an adapter's
// term, a sum over pieces): a 256 x 256 tile of
//     NT:  C[i][j] = sum_k L[i][k] R[j][k]      R row-major [cols][contraction]
//     NN:  C[i][j] = sum_k L[i][k] R[k][j]      R row-major [contraction][cols]
//
//  * 512 threads, 8 waves as 2 x 4, each 128 x 64 of fp32 accumulators;
//    contraction step 64, both operands global -> LDS by DMA one step ahead
//    (two stages of 32 KB each).
//  * LDS rows of 128 bytes (L, and R of NT) and of 512 bytes (R of NN) with
//    their 16-byte chunks XOR-swizzled by row; NN reads its right operand with
//    the transposing LDS load, so that neither form needs a transposed copy.
//  * R is the matrix instruction's left operand, so a lane's accumulators run
//    along a row of C: lane l holds row 32 i + l % 32 of its wave's block and,
//    in element e of acc[i][j], column 32 j + 8 (e / 4) + 4 (l / 32) + e % 4.
//    Sums over a row are then sums within a lane and one exchange.
//  * Operands of sub-step s + 1 are read while sub-step s multiplies, and the
//    last products of a step run after its barrier, over the next step's first
//    reads.
#pragma once

#include "common.h"
#include "lds_dma.h"
#include "tile.h"

namespace qlora {
namespace gemm16 {

typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));

constexpr int kBM = 256, kBN = 256, kBK = 64;
constexpr int kThreads = 512;
constexpr int kStage = 256 * 64 * 2;
constexpr int kLds = 4 * kStage;
constexpr int kXcds = 8;
constexpr int kBand = 4;   // tile rows of a band: an XCD's tiles share rows of L and columns of R in its L2

// 512-byte rows (256 bf16): chunk c of row r at c ^ g(r).
__device__ __forceinline__ int swz512(int row, int chunk) {
  return row * 512 + 16 * (chunk ^ (((row & 3) << 2) | ((row >> 2) & 3)));
}

// Tile `id` of `tiles` (trows x tcols): workgroups go to the 8 XCDs in turn,
// each XCD has a run of consecutive tiles, numbered in bands of kBand tile rows
// column by column.  The count may be smaller than the grid (it may be known on
// the device alone); false: no tile for this workgroup.
__device__ __forceinline__ bool place(int id, int trows, int tcols, int &tr, int &tc) {
  const int tiles = trows * tcols;
  if (id >= tiles) return false;
  const int each = tiles / kXcds, over = tiles % kXcds;
  const int x = id % kXcds, y = id / kXcds;
  const int lid = x * each + min(x, over) + y;
  const int band = lid / (kBand * tcols);
  const int h = min(kBand, trows - band * kBand);
  const int j = lid - band * kBand * tcols;
  tc = j / h;
  tr = band * kBand + j % h;
  return true;
}

struct Frag {
  bf16x8_t a[4], b[2];
};

struct Offsets {
  uint32_t xo[4], wo[4], to[2][2];
};

__device__ __forceinline__ Offsets offsets() {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 2, wn = wave & 3;
  const int lr = lane & 31, lh = lane >> 5;
  Offsets o;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    o.xo[s] = static_cast<uint32_t>(swz128(128 * wm + lr, 2 * s + lh));
    o.wo[s] = static_cast<uint32_t>(swz128(64 * wn + lr, 2 * s + lh));
  }
  // [64 contraction][256 columns] stage: lanes 16 G .. 16 G + 15 get columns
  // 64 wn + 32 j + 16 (G % 2) .. +15 of rows 8 (G / 2) + 4 h .. +3 (+ 16 s);
  // source lane t points at row t / 4 and columns 4 (t % 4) .. +3 of them.
  const int t = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      o.to[j][h] = static_cast<uint32_t>(
          swz512(8 * (g >> 1) + 4 * h + (t >> 2), 8 * wn + 4 * j + 2 * (g & 1) + ((t & 3) >> 1)) + 8 * (t & 1));
  return o;
}

__device__ __forceinline__ bf16x4_t ds_tr16(const uint8_t *p) {
  typedef __attribute__((address_space(3))) bf16x4_t lds_t;
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_t *)((__attribute__((address_space(3))) uint8_t *)(p)));
}

template <bool kNN>
__device__ __forceinline__ void load_frag(Frag &f, const uint8_t *xs, const uint8_t *ws, const Offsets &o, int s) {
  auto ld_a = [&](int i) { f.a[i] = *reinterpret_cast<const bf16x8_t *>(xs + o.xo[s] + 4096 * i); };
  auto ld_b = [&](int j) {
    if (!kNN) {
      f.b[j] = *reinterpret_cast<const bf16x8_t *>(ws + o.wo[s] + 4096 * j);
    } else {
      const bf16x4_t lo = ds_tr16(ws + o.to[j][0] + 8192 * s);
      const bf16x4_t hi = ds_tr16(ws + o.to[j][1] + 8192 * s);
      f.b[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  };
  ld_a(0);
  ld_b(0);
  ld_b(1);
  ld_a(1);
  ld_a(2);
  ld_a(3);
}

template <int i0, int i1>
__device__ __forceinline__ void mfma_rows(const Frag &f, f32x16_t (&acc)[4][2]) {
#pragma unroll
  for (int i = i0; i < i1; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
}

__device__ __forceinline__ void clear(f32x16_t (&acc)[4][2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
}

// This thread's place in the four 1 KB DMA instructions of a stage with
// 128-byte rows: row(j) of the tile, and the chunk that lands at its position.
struct RowDma {
  int wave, lane;
  __device__ __forceinline__ RowDma() : wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), lane(threadIdx.x & 63) {}
  __device__ __forceinline__ int row(int j) const { return (wave * 4 + j) * 8 + (lane >> 3); }
  __device__ __forceinline__ int chunk(int j) const {
    const int r = row(j);
    return (lane & 7) ^ ((r & 7) ^ ((r >> 3) & 1));
  }
  // Of a [64][256] stage.
  __device__ __forceinline__ int krow(int j) const { return 2 * (wave * 4 + j) + (lane >> 5); }
  __device__ __forceinline__ int kchunk(int j) const {
    const int r = krow(j);
    return (lane & 31) ^ (((r & 3) << 2) | ((r >> 2) & 3));
  }
};

// One tile.  smem: kLds bytes.  lrow(row of the tile) gives a row of L (in
// range: rows past the end repeat a valid one and are never stored); both
// operands' byte offsets from their bases stay below 2^32.  NT: R's rows c0 ..
// c0 + 255 clamped to rlast; NN: R's columns likewise (chunks of 8, rlast + 1 a
// multiple of 8) and contraction rows past klast repeat it (L holds zeros there).
// KT >= 1 steps of 64.  Ends with a barrier: smem is free.
template <bool kNN, class LRow>
__device__ __forceinline__ void tile(uint8_t *smem, const uint16_t *L, uint32_t ldl, LRow lrow, const uint16_t *R,
                                     uint32_t ldr, int c0, int rlast, int klast, int KT, f32x16_t (&acc)[4][2]) {
  uint8_t *const sX[2] = {smem, smem + kStage};
  uint8_t *const sW[2] = {smem + 2 * kStage, smem + 3 * kStage};
  const RowDma d;
  uint32_t lo[4], ro[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    lo[j] = static_cast<uint32_t>(lrow(d.row(j))) * ldl * 2 + 16 * d.chunk(j);
    if (kNN)
      ro[j] = 2 * static_cast<uint32_t>(min(c0 + 8 * d.kchunk(j), rlast - 7));
    else
      ro[j] = static_cast<uint32_t>(min(c0 + d.row(j), rlast)) * ldr * 2 + 16 * d.chunk(j);
  }
  const uint32_t lds0 = lds_addr(smem);
  auto dma_l = [&](int st, int kt) __attribute__((always_inline)) {
    const uint16_t *base = L + static_cast<int64_t>(kBK) * kt;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      dma16(base, lo[j], __builtin_amdgcn_readfirstlane(lds0 + st * kStage + (d.wave * 4 + j) * 1024));
  };
  auto dma_r = [&](int st, int kt) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + (2 + st) * kStage + d.wave * 4096;
    if (kNN) {
      const uint16_t *base = R + static_cast<int64_t>(kBK) * kt * ldr;
      const int last = klast - kBK * kt;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        dma16(base, static_cast<uint32_t>(min(d.krow(j), last)) * ldr * 2 + ro[j], __builtin_amdgcn_readfirstlane(dst + j * 1024));
    } else {
      const uint16_t *base = R + static_cast<int64_t>(kBK) * kt;
#pragma unroll
      for (int j = 0; j < 4; ++j) dma16(base, ro[j], __builtin_amdgcn_readfirstlane(dst + j * 1024));
    }
  };
  const Offsets ops = offsets();
  clear(acc);
  dma_l(0, 0);
  dma_r(0, 0);
  raw_barrier<wait_imm(0, 0)>();
  Frag fa, fb;
#pragma unroll
  for (int i = 0; i < 4; ++i) fb.a[i] = bf16x8_t{};
#pragma unroll
  for (int j = 0; j < 2; ++j) fb.b[j] = bf16x8_t{};
  auto step = [&](int cur, int kt) __attribute__((always_inline)) {
    const uint8_t *xs = sX[cur];
    const uint8_t *ws = sW[cur];
    load_frag<kNN>(fa, xs, ws, ops, 0);
    __builtin_amdgcn_sched_barrier(0);
    mfma_rows<2, 3>(fb, acc);
    if (kt + 1 < KT) dma_l(cur ^ 1, kt + 1);
    __builtin_amdgcn_sched_barrier(0);
    mfma_rows<3, 4>(fb, acc);
    if (kt + 1 < KT) dma_r(cur ^ 1, kt + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      Frag &now = (s & 1) ? fb : fa;
      Frag &nxt = (s & 1) ? fa : fb;
      mfma_rows<0, 1>(now, acc);
      __builtin_amdgcn_sched_barrier(0);
      if (s < 3) load_frag<kNN>(nxt, xs, ws, ops, s + 1);
      mfma_rows<1, 2>(now, acc);
      __builtin_amdgcn_sched_barrier(0);
      if (s < 3) mfma_rows<2, 4>(now, acc);
      __builtin_amdgcn_sched_barrier(0);
    }
    raw_barrier<wait_imm(0, 0)>();
  };
  int kt = 0;
  for (; kt + 2 <= KT; kt += 2) {
    step(0, kt);
    step(1, kt + 1);
  }
  if (kt < KT) step(0, kt);
  mfma_rows<2, 4>(fb, acc);   // held back by the last step
}

// The wave's 128 x 64 block as bf16 by way of its own 16 KB of smem (free), in
// whole 128-byte row segments: put(row of the tile, column of the tile, 16 bytes).
template <class Put>
__device__ __forceinline__ void store_bf16(const f32x16_t (&acc)[4][2], uint8_t *smem, Put put) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave >> 2, wn = wave & 3, lr = lane & 31, lh = lane >> 5;
  uint8_t *region = smem + wave * 16384;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int rr = 32 * i + lr;
        const uint2 v = make_uint2(pack_bf16x2(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                                   pack_bf16x2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]));
        *reinterpret_cast<uint2 *>(region + rr * 128 + 16 * ((4 * j + q) ^ (rr & 7)) + 8 * lh) = v;
      }
  __builtin_amdgcn_s_waitcnt(wait_imm(63, 0));
  __builtin_amdgcn_wave_barrier();
#pragma unroll 4
  for (int t = 0; t < 16; ++t) {
    const int rr = t * 8 + (lane >> 3), c = lane & 7;
    const uint4 v = *reinterpret_cast<const uint4 *>(region + rr * 128 + 16 * (c ^ (rr & 7)));
    put(128 * wm + rr, 64 * wn + 8 * c, v);
  }
}

}  // namespace gemm16
}  // namespace qlora
