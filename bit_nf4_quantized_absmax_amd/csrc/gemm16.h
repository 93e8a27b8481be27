// The bf16 product of two matrices on gfx950's matrix instructions, as a device
// function whose callers add what follows it (a row's softmax, an adapter's
// term, a sum over pieces): a tile of
//     NT:  C[i][j] = sum_k L[i][k] R[j][k]      R row-major [cols][contraction]
//     NN:  C[i][j] = sum_k L[i][k] R[k][j]      R row-major [contraction][cols]
//
//  * Tiles of kWM x kWN waves of 32 kFM x 32 kFN fp32 accumulators each: Big, 256 x
//    256 of 8 waves, and Mid and Deep, 128 x 128 of 4, for products with too few
//    Big tiles to fill the chip.
//  * Contraction step 64, both operands global -> LDS by DMA one step ahead (two
//    stages of each; a compute unit holds two Mid workgroups, which hide each other's
//    waits), in Deep, for a workgroup that is alone on its compute unit, two ahead.
//  * LDS rows of 128 bytes (L, and R of NT) and of 2 BN bytes (R of NN) with
//    their 16-byte chunks XOR-swizzled by row; NN reads its right operand with
//    the transposing LDS load, so that neither form needs a transposed copy.
//  * R is the matrix instruction's left operand, so a lane's accumulators run
//    along a row of C: lane l holds row 32 i + l % 32 of its wave's block and,
//    in element e of acc[i][j], column 32 j + 8 (e / 4) + 4 (l / 32) + e % 4.
//    Sums over a row are then sums within a lane and one exchange.
//  * Operands of sub-step s + 1 are read while sub-step s multiplies, and the
//    last products of a step run after its barrier, over the next step's first
//    reads.
//
// Bound by the matrix pipes beside the LDS that feeds them: large products reach
// 1.15 to 1.25 PFLOP/s (8192 x 4096 x 11008: 600 us at its best, 690 in the middle), where
// the library's plain product of 8192^3 reaches 1.42 on the same card.
#pragma once

#include "common.h"
#include "lds_dma.h"
#include "tile.h"

namespace qlora {
namespace gemm16 {

typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));

constexpr int kBK = 64;
constexpr int kXcds = 8;
constexpr int kBand = 4;   // tile rows of a band: an XCD's tiles share rows of L and columns of R in its L2 (2, 8 and 16: 1 to 3 % longer)

template <int kWM_, int kWN_, int kFM_, int kFN_, int kStages_ = 2>
struct Shape {
  static constexpr int kStages = kStages_;
  static constexpr int kWM = kWM_, kWN = kWN_, kFM = kFM_, kFN = kFN_;
  static constexpr int kBM = 32 * kFM * kWM, kBN = 32 * kFN * kWN;
  static constexpr int kWaves = kWM * kWN, kThreads = 64 * kWaves;
  static constexpr int kStageL = kBM * 128, kStageR = kBN * 128;
  static constexpr int kLds = kStages * (kStageL + kStageR);
  static constexpr int kWaveRows = 32 * kFM, kWaveCols = 32 * kFN;
  static constexpr int kDmaL = kBM / 8 / kWaves, kDmaR = kBN / 8 / kWaves;   // 1 KB instructions a wave and stage
  static_assert(kLds >= kWaves * kWaveRows * kWaveCols * 2, "the tile in bf16 fits the stages");
};
using Big = Shape<2, 4, 4, 2>;
using Mid = Shape<2, 2, 2, 2>;
using Deep = Shape<2, 2, 2, 2, 3>;

// Whether a product takes Mid tiles, by the rounds that its tiles make of the 256
// compute units.  A round of Big tiles is four Mid tiles' work; two Mid
// workgroups of a unit take 2.7 such units of time and one alone 1.7 (measured, us, Big
// and Mid: 2048 x 4096 x 4096 121 and 98, 1024 x 4096 x 4096 123 and 83, 777 x
// 5000 x 1088 54 and 45, 300 x 32000 x 4096 280 and 302, 300 x 50001 x 1088 118 and 124).
inline bool use_mid(int64_t rows, int64_t cols) {
  const int64_t big = ((rows + 255) / 256) * ((cols + 255) / 256), mid = ((rows + 127) / 128) * ((cols + 127) / 128);
  return (mid <= 256 ? 17 : 27 * ((mid + 511) / 512)) < 40 * ((big + 255) / 256);
}

// Deep tiles instead of Mid ones where every tile has a compute unit to itself (the layer with
// adapters, us, Mid with its contraction split for 512 workgroups and Deep for 256: 256 x
// 4096 x 4096 52 and 45, 192 x 4096 x 4096 50 and 44, 1024 x 4096 x 4096 68 and 65, 105 x 3232 x
// 10944 61 and 56; four stages as three; 300 Deep tiles take two rounds: 777 x 5000 x
// 1088 40 and 54).
inline bool use_deep(int64_t rows, int64_t cols) { return ((rows + 127) / 128) * ((cols + 127) / 128) <= 256; }

// Rows of 2 BN bytes: chunk c of row r at c ^ g(r).
template <class S>
__device__ __forceinline__ int swz_wide(int row, int chunk) {
  return row * 2 * S::kBN + 16 * (chunk ^ (((row & 3) << 2) | ((row >> 2) & 3)));
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

template <class S>
using Acc = f32x16_t[S::kFM][S::kFN];

template <class S>
struct Frag {
  bf16x8_t a[S::kFM], b[S::kFN];
};

template <class S>
struct Offsets {
  uint32_t xo[4], wo[4], to[S::kFN][2];
};

// This thread's wave in the tile.
template <class S>
struct Place {
  int wave, lane, wm, wn, lr, lh;
  __device__ __forceinline__ Place()
      : wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), lane(threadIdx.x & 63), wm(wave / S::kWN), wn(wave % S::kWN),
        lr(lane & 31), lh(lane >> 5) {}
  __device__ __forceinline__ int row0() const { return S::kWaveRows * wm; }
  __device__ __forceinline__ int col0() const { return S::kWaveCols * wn; }
};

template <class S>
__device__ __forceinline__ Offsets<S> offsets(const Place<S> &p) {
  Offsets<S> o;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    o.xo[s] = static_cast<uint32_t>(swz128(p.row0() + p.lr, 2 * s + p.lh));
    o.wo[s] = static_cast<uint32_t>(swz128(p.col0() + p.lr, 2 * s + p.lh));
  }
  // [64 contraction][BN columns] stage: lanes 16 G .. 16 G + 15 get columns
  // 32 j + 16 (G % 2) .. +15 of the wave's and rows 8 (G / 2) + 4 h .. +3 (+ 16 s);
  // source lane t points at row t / 4 and columns 4 (t % 4) .. +3 of them.
  const int t = p.lane & 15, g = p.lane >> 4;
#pragma unroll
  for (int j = 0; j < S::kFN; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      o.to[j][h] = static_cast<uint32_t>(
          swz_wide<S>(8 * (g >> 1) + 4 * h + (t >> 2), p.col0() / 8 + 4 * j + 2 * (g & 1) + ((t & 3) >> 1)) + 8 * (t & 1));
  return o;
}

__device__ __forceinline__ bf16x4_t ds_tr16(const uint8_t *p) {
  typedef __attribute__((address_space(3))) bf16x4_t lds_t;
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_t *)((__attribute__((address_space(3))) uint8_t *)(p)));
}

template <class S, bool kNN>
__device__ __forceinline__ void load_frag(Frag<S> &f, const uint8_t *xs, const uint8_t *ws, const Offsets<S> &o, int s) {
  auto ld_a = [&](int i) { f.a[i] = *reinterpret_cast<const bf16x8_t *>(xs + o.xo[s] + 4096 * i); };
  auto ld_b = [&](int j) {
    if (!kNN) {
      f.b[j] = *reinterpret_cast<const bf16x8_t *>(ws + o.wo[s] + 4096 * j);
    } else {
      const bf16x4_t lo = ds_tr16(ws + o.to[j][0] + 32 * S::kBN * s);
      const bf16x4_t hi = ds_tr16(ws + o.to[j][1] + 32 * S::kBN * s);
      f.b[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  };
  ld_a(0);
#pragma unroll
  for (int j = 0; j < S::kFN; ++j) ld_b(j);
#pragma unroll
  for (int i = 1; i < S::kFM; ++i) ld_a(i);
}

template <class S, int i0, int i1>
__device__ __forceinline__ void mfma_rows(const Frag<S> &f, Acc<S> &acc) {
#pragma unroll
  for (int i = i0; i < i1; ++i)
#pragma unroll
    for (int j = 0; j < S::kFN; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
}

template <class S>
__device__ __forceinline__ void clear(Acc<S> &acc) {
#pragma unroll
  for (int i = 0; i < S::kFM; ++i)
#pragma unroll
    for (int j = 0; j < S::kFN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
}

// One tile.  smem: S::kLds bytes.  lrow(row of the tile) gives a row of L (in
// range: rows past the end repeat a valid one and are never stored); both
// operands' byte offsets from their bases stay below 2^32.  NT: R's rows c0 ..
// clamped to rlast; NN: R's columns likewise (chunks of 8, rlast + 1 a
// multiple of 8) and contraction rows past klast repeat it (L holds zeros there).
// KT >= 1 steps of 64.  Ends with a barrier: smem is free.
template <class S, bool kNN, class LRow>
__device__ __forceinline__ void tile(uint8_t *smem, const uint16_t *L, uint32_t ldl, LRow lrow, const uint16_t *R,
                                     uint32_t ldr, int c0, int rlast, int klast, int KT, Acc<S> &acc) {
  const Place<S> p;
  // A DMA instruction fills 1 KB: 8 rows of 128 bytes, or 512 / BN of the wide ones;
  // a lane fetches the chunk that belongs at its position.
  uint32_t lo[S::kDmaL], ro[S::kDmaR];
  auto chunk8 = [](int row, int lane) { return (lane & 7) ^ ((row & 7) ^ ((row >> 3) & 1)); };
  constexpr int kWideLanes = S::kBN / 8;             // lanes of a wide row
  auto wide_row = [&](int j) { return (64 / kWideLanes) * (p.wave * S::kDmaR + j) + p.lane / kWideLanes; };
#pragma unroll
  for (int j = 0; j < S::kDmaL; ++j) {
    const int row = (p.wave * S::kDmaL + j) * 8 + (p.lane >> 3);
    lo[j] = static_cast<uint32_t>(lrow(row)) * ldl * 2 + 16 * chunk8(row, p.lane);
  }
#pragma unroll
  for (int j = 0; j < S::kDmaR; ++j) {
    if (kNN) {
      const int row = wide_row(j);
      const int chunk = (p.lane % kWideLanes) ^ (((row & 3) << 2) | ((row >> 2) & 3));
      ro[j] = 2 * static_cast<uint32_t>(min(c0 + 8 * chunk, rlast - 7));
    } else {
      const int row = (p.wave * S::kDmaR + j) * 8 + (p.lane >> 3);
      ro[j] = static_cast<uint32_t>(min(c0 + row, rlast)) * ldr * 2 + 16 * chunk8(row, p.lane);
    }
  }
  const uint32_t lds0 = lds_addr(smem);
  auto dma_l = [&](int st, int kt) __attribute__((always_inline)) {
    const uint16_t *base = L + static_cast<int64_t>(kBK) * kt;
#pragma unroll
    for (int j = 0; j < S::kDmaL; ++j)
      dma16(base, lo[j], __builtin_amdgcn_readfirstlane(lds0 + st * S::kStageL + (p.wave * S::kDmaL + j) * 1024));
  };
  auto dma_r = [&](int st, int kt) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + S::kStages * S::kStageL + st * S::kStageR + p.wave * S::kDmaR * 1024;
    if (kNN) {
      const uint16_t *base = R + static_cast<int64_t>(kBK) * kt * ldr;
      const int last = klast - kBK * kt;
#pragma unroll
      for (int j = 0; j < S::kDmaR; ++j)
        dma16(base, static_cast<uint32_t>(min(wide_row(j), last)) * ldr * 2 + ro[j], __builtin_amdgcn_readfirstlane(dst + j * 1024));
    } else {
      const uint16_t *base = R + static_cast<int64_t>(kBK) * kt;
#pragma unroll
      for (int j = 0; j < S::kDmaR; ++j) dma16(base, ro[j], __builtin_amdgcn_readfirstlane(dst + j * 1024));
    }
  };
  const Offsets<S> ops = offsets<S>(p);
  clear<S>(acc);
  constexpr int kDma = S::kDmaL + S::kDmaR, kAhead = S::kStages - 1;   // steps that are asked for ahead
  static_assert(kAhead <= 2, "the waits below");
#pragma unroll
  for (int st = 0; st < kAhead; ++st)
    if (st < KT) {
      dma_l(st, st);
      dma_r(st, st);
    }
  // Waits until a step has landed, `behind` of the steps after it being asked for.
  auto landed = [&](int behind) __attribute__((always_inline)) {
    if (kAhead > 1 && behind >= 1)
      raw_barrier<wait_imm(kDma, 0)>();
    else
      raw_barrier<wait_imm(0, 0)>();
  };
  landed(min(kAhead, KT) - 1);
  Frag<S> fa, fb;
#pragma unroll
  for (int i = 0; i < S::kFM; ++i) fb.a[i] = bf16x8_t{};
#pragma unroll
  for (int j = 0; j < S::kFN; ++j) fb.b[j] = bf16x8_t{};
  constexpr int kHeld = S::kFM / 2;                  // row fragments of a step's last products held back over its barrier
  auto step = [&](int cur, int kt) __attribute__((always_inline)) {
    const uint8_t *xs = smem + cur * S::kStageL;
    const uint8_t *ws = smem + S::kStages * S::kStageL + cur * S::kStageR;
    const int fill = kAhead == 1 ? cur ^ 1 : cur == 0 ? kAhead : cur - 1;
    load_frag<S, kNN>(fa, xs, ws, ops, 0);
    __builtin_amdgcn_sched_barrier(0);
    mfma_rows<S, kHeld, kHeld + (S::kFM - kHeld) / 2>(fb, acc);
    if (kt + kAhead < KT) dma_l(fill, kt + kAhead);
    __builtin_amdgcn_sched_barrier(0);
    mfma_rows<S, kHeld + (S::kFM - kHeld) / 2, S::kFM>(fb, acc);
    if (kt + kAhead < KT) dma_r(fill, kt + kAhead);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      Frag<S> &now = (s & 1) ? fb : fa;
      Frag<S> &nxt = (s & 1) ? fa : fb;
      mfma_rows<S, 0, kHeld / 2>(now, acc);
      __builtin_amdgcn_sched_barrier(0);
      if (s < 3) load_frag<S, kNN>(nxt, xs, ws, ops, s + 1);
      mfma_rows<S, kHeld / 2, kHeld>(now, acc);
      __builtin_amdgcn_sched_barrier(0);
      if (s < 3) mfma_rows<S, kHeld, S::kFM>(now, acc);
      __builtin_amdgcn_sched_barrier(0);
    }
    landed(min(kt + kAhead, KT - 1) - (kt + 1));
  };
  int kt = 0;
  if constexpr (S::kStages == 2) {
    for (; kt + 2 <= KT; kt += 2) {
      step(0, kt);
      step(1, kt + 1);
    }
    if (kt < KT) step(0, kt);
  } else {
    int cur = 0;
#pragma unroll 1
    for (; kt < KT; ++kt) {
      step(cur, kt);
      cur = cur == kAhead ? 0 : cur + 1;
    }
  }
  mfma_rows<S, kHeld, S::kFM>(fb, acc);   // held back by the last step
}

// The wave's block as bf16 by way of its own part of smem (free), in whole row
// segments of it: put(row of the tile, column of the tile, 16 bytes).
template <class S, class Put>
__device__ __forceinline__ void store_bf16(const Acc<S> &acc, uint8_t *smem, Put put) {
  static_assert(S::kWaveCols == 64, "row segments of 128 bytes");
  const Place<S> p;
  uint8_t *region = smem + p.wave * S::kWaveRows * 128;
#pragma unroll
  for (int i = 0; i < S::kFM; ++i)
#pragma unroll
    for (int j = 0; j < S::kFN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int rr = 32 * i + p.lr;
        const uint2 v = make_uint2(pack_bf16x2(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                                   pack_bf16x2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]));
        *reinterpret_cast<uint2 *>(region + rr * 128 + 16 * ((4 * j + q) ^ (rr & 7)) + 8 * p.lh) = v;
      }
  __builtin_amdgcn_s_waitcnt(wait_imm(63, 0));
  __builtin_amdgcn_wave_barrier();
#pragma unroll 4
  for (int t = 0; t < S::kWaveRows / 8; ++t) {
    const int rr = t * 8 + (p.lane >> 3), c = p.lane & 7;
    const uint4 v = *reinterpret_cast<const uint4 *>(region + rr * 128 + 16 * (c ^ (rr & 7)));
    put(p.row0() + rr, p.col0() + 8 * c, v);
  }
}

}  // namespace gemm16
}  // namespace qlora
