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
//  * Operands of sub-step s + 1 are read while sub-step s multiplies; part of
//    a step's last products run after its barrier, over the first reads of
//    the next step.
//  * The LoRA term is one (r <= 64) or two more steps on bf16 MFMA into the
//    same accumulators.  At r = 64 its rows are as long as a slab's, and the
//    step is one more of the DMA pipeline.
//  * A workgroup takes tiles until none is left; the last step of a tile
//    already fetches the first of the next, and the tile is stored over it.
//    W is the matrix instruction's left operand, so that a lane's
//    accumulators run along a row of Y: two half-wave swaps make 16 bytes of
//    them, which cross the wave's own part of a free stage.
//
// 8192 x 11008 x 4096 with r = 64: 205 to 230 us, 3.2 to 3.6 PFLOP/s, 0.62 to 0.70
// of four times what a large bf16 product reaches here, the matrix pipes busy 45 %
// of the clocks.  No part of it is the bound by itself: of 227 us, 163 remain
// without the fetch, 167 without the products and 72 without both (operand reads,
// barriers, stores): fetch and products overlap by a third, since a step's barrier
// waits for the fetch that the step itself issued.  The 1376 tiles are six
// rounds of the 256 compute units, the last of 96 tiles.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "lds_dma.h"
#include "tile.h"

namespace qlora {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kMxMmThreads = 512;
constexpr int kMxBand = 4;   // tile rows of a band (see Tiles); 8192 x 11008 x 4096: 206 us, in bands of one 218
constexpr int kCUs = 256;
constexpr int kXcds = 8;

struct Mx4Args {
  const uint8_t *xc, *xs, *wc, *ws;
  const uint16_t *T, *B;
  uint16_t *Y;
  int M, N, r;
  int KT;            // slabs
  int trows, tcols;
  float *part;       // split: partial tiles [splits][tiles], else unused
  int splits;
};

// The tiles of a workgroup.  Workgroups go to the 8 XCDs in turn; each XCD has
// a run of consecutive tiles and its workgroups take them in turn (as many
// tiles as workgroups: one each).  Tiles are numbered in bands of kMxBand tile
// rows, column by column, so that the tiles an XCD has in work share rows of
// X and of W in its L2.
struct Tiles {
  int next, end, step;
  __device__ __forceinline__ Tiles(int n, int e, int s) : next(n), end(e), step(s) {}
  __device__ __forceinline__ explicit Tiles(int tiles) {
    const int x = blockIdx.x % kXcds, each = tiles / kXcds, over = tiles % kXcds;
    const int begin = x * each + min(x, over);
    next = begin + blockIdx.x / kXcds;
    end = begin + each + (x < over ? 1 : 0);
    step = (gridDim.x - x + kXcds - 1) / kXcds;   // workgroups of this XCD
  }
  __device__ __forceinline__ static void place(const Mx4Args &a, int id, int bm, int bn, int &m0, int &n0) {
    const int band = id / (kMxBand * a.tcols);
    const int h = min(kMxBand, a.trows - band * kMxBand);
    const int j = id - band * kMxBand * a.tcols;
    n0 = j / h * bn;
    m0 = (band * kMxBand + j % h) * bm;
  }
};

// kRows rows of 128 bytes, `pitch` apart, from src (the tile's first) into a
// swizzled stage at LDS address `stage`; rows past `last` repeat it (their
// results are not stored).
template <int kRows>
__device__ __forceinline__ void dma_rows(uint32_t stage, const uint8_t *src, uint32_t pitch, int last, int wave, int lane) {
#pragma unroll
  for (int j = 0; j < kRows / 64; ++j) {
    const int u = wave * (kRows / 64) + j;
    const int row = u * 8 + (lane >> 3);
    const int chunk = (lane & 7) ^ ((row & 7) ^ ((row >> 3) & 1));
    dma16(src, static_cast<uint32_t>(min(row, last)) * pitch + chunk * 16,
          __builtin_amdgcn_readfirstlane(stage + u * 1024));
  }
}

// Scales of rows 32 u .. 32 u + 31: 8 bytes a row.
__device__ __forceinline__ void dma_scales(uint32_t stage, const uint8_t *src, int last, int u, int lane) {
  dma4(src, min(32 * u + (lane >> 1), last) * 8 + 4 * (lane & 1), __builtin_amdgcn_readfirstlane(stage + u * 256));
}

__device__ __forceinline__ i32x8_t widen(i32x4_t v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }

// One 32 x 32 x 64 product under the scales in byte kByte of sa and sb.
template <int kByte>
__device__ __forceinline__ f32x16_t mfma4(i32x4_t a, i32x4_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), widen(b), c, 4, 4, kByte, static_cast<int>(sa), kByte,
                                                         static_cast<int>(sb));
}

// Operands of a sub-step (a: X or T rows, b: W or B rows) and a step's scales.
template <int kFM, int kFN>
struct Ops {
  i32x4_t a[kFM], b[kFN];
};
template <int kFM, int kFN>
struct Scales {
  uint2 a[kFM], b[kFN];
};

// Product of one pair of fragments in sub-step s under scale words sa, sb.
template <bool kLora>
__device__ __forceinline__ f32x16_t mul1(i32x4_t a, i32x4_t b, uint32_t sa, uint32_t sb, int s, f32x16_t acc) {
  if constexpr (kLora)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, b), __builtin_bit_cast(bf16x8_t, a), acc, 0, 0,
                                                   0);
  return (s & 1) ? mfma4<2>(b, a, acc, sb, sa) : mfma4<0>(b, a, acc, sb, sa);
}

// Products of row fragments i0 .. i1 - 1 of sub-step s.
template <int i0, int i1, bool kLora, int kFM, int kFN>
__device__ __forceinline__ void mul(const Ops<kFM, kFN> &o, const Scales<kFM, kFN> &sc, int s, f32x16_t (&acc)[kFM][kFN]) {
#pragma unroll
  for (int i = i0; i < i1; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j)
      acc[i][j] = mul1<kLora>(o.a[i], o.b[j], s < 2 ? sc.a[i].x : sc.a[i].y, s < 2 ? sc.b[j].x : sc.b[j].y, s, acc[i][j]);
}

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

// Swaps the upper half-wave of a with the lower one of b.
__device__ __forceinline__ void swap_halves(uint32_t &a, uint32_t &b) {
  typedef unsigned int pair_t __attribute__((ext_vector_type(2)));
  const pair_t r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

typedef uint4 __attribute__((aligned(2))) uint4_any;   // rows of an odd N start anywhere

}  // namespace

// kPiped: r == 64, the LoRA step runs in the pipeline.  kSplit: a workgroup has
// one tile and a part of the contraction, and leaves its fp32 sums (the last
// part's with the LoRA term) for k_mx4_join.  kBf16 (with kSplit): X and W are
// bf16, every step is one of 64 columns on bf16 MFMA and there are no scales.
template <int kFM, int kFN, bool kPiped, bool kSplit, bool kBf16 = false>
__global__ __launch_bounds__(kMxMmThreads) void k_mx4_matmul(const Mx4Args args) {
  constexpr int kBM = 64 * kFM, kBN = 128 * kFN;
  constexpr int kHold = kFM / 2;                 // row fragments whose last products run after the barrier
  // Stages: X codes | W codes (two each, a power of two apart) | scales.
  constexpr uint32_t kStX = kBM * 128, kStW = kBN * 128, kOffW = 2 * kStX, kOffS = kOffW + 2 * kStW;
  constexpr uint32_t kStS = (kBM + kBN) * 8;
  static_assert((kOffW & kStX) == 0 && (kOffW & kStW) == 0 && (kOffS % kStS) == 0, "stages toggle by one bit");
  __shared__ __attribute__((aligned(128))) uint8_t smem[kOffS + 2 * kStS];

  const int M = args.M, N = args.N, r = args.r, KT = args.KT;
  const int tile = kSplit ? blockIdx.x / args.splits : 0, split = kSplit ? blockIdx.x % args.splits : 0;
  const int k0 = kSplit ? KT * split / args.splits : 0, k1 = kSplit ? KT * (split + 1) / args.splits : KT;
  const bool last = !kSplit || split == args.splits - 1;   // takes the LoRA steps
  const int steps = k1 + (kPiped && last ? 1 : 0);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int lr = lane & 31, lh = lane >> 5;
  const uint32_t base = lds_addr(smem);

  Tiles tiles(args.trows * args.tcols);
  if constexpr (kSplit) tiles = Tiles{tile, tile + 1, 1};
  if (tiles.next >= tiles.end) return;   // the whole workgroup

  auto dma = [&](uint32_t st, int m0, int n0, int kt, int part) __attribute__((always_inline)) {
    const uint32_t x = base + (st ? kStX : 0), w = base + kOffW + (st ? kStW : 0), sc = base + kOffS + (st ? kStS : 0);
    const int lastm = M - 1 - m0, lastn = N - 1 - n0;
    if (kPiped && kt == KT) {
      if (part & 1) dma_rows<kBM>(x, reinterpret_cast<const uint8_t *>(args.T) + static_cast<int64_t>(m0) * 128, 128, lastm, wave, lane);
      if (part & 2) dma_rows<kBN>(w, reinterpret_cast<const uint8_t *>(args.B) + static_cast<int64_t>(n0) * 128, 128, lastn, wave, lane);
      return;
    }
    const uint32_t pitch = static_cast<uint32_t>(KT) * 128;
    if (part & 1) dma_rows<kBM>(x, args.xc + static_cast<int64_t>(m0) * pitch + kt * 128, pitch, lastm, wave, lane);
    if (part & 2) dma_rows<kBN>(w, args.wc + static_cast<int64_t>(n0) * pitch + kt * 128, pitch, lastn, wave, lane);
    if (!kBf16 && (part & 1))
#pragma unroll
    for (int u = wave; u < (kBM + kBN) / 32; u += 8) {
      if (u < kBM / 32)
        dma_scales(sc, args.xs + (static_cast<int64_t>(kt) * M + m0) * 8, lastm, u, lane);
      else
        dma_scales(sc + kBM * 8, args.ws + (static_cast<int64_t>(kt) * N + n0) * 8, lastn, u - kBM / 32, lane);
    }
  };
  // Operand reads of sub-step 0 of the current stage; fragment i adds 4096 i,
  // sub-step s turns bits 5 and 6 (chunk 2 s + lh of the swizzled row).
  uint32_t xo = static_cast<uint32_t>(swz128(32 * kFM * wm + lr, lh));
  uint32_t wo = kOffW + static_cast<uint32_t>(swz128(32 * kFN * wn + lr, lh));
  uint32_t so = kOffS + (32 * kFM * wm + lr) * 8, to = kOffS + (kBM + 32 * kFN * wn + lr) * 8;

  f32x16_t acc[kFM][kFN];
  Ops<kFM, kFN> fa, fb;
  Scales<kFM, kFN> sc;
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kFM; ++i)
#pragma unroll
      for (int j = 0; j < kFN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    // the first step has no products held back: zeros under the smallest scale
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
      fb.a[i] = i32x4_t{0, 0, 0, 0};
      sc.a[i] = make_uint2(0, 0);
    }
#pragma unroll
    for (int j = 0; j < kFN; ++j) {
      fb.b[j] = i32x4_t{0, 0, 0, 0};
      sc.b[j] = make_uint2(0, 0);
    }
  };
  auto read = [&](Ops<kFM, kFN> &o, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kFN; ++j) o.b[j] = *reinterpret_cast<const i32x4_t *>(smem + (wo ^ (32u * s)) + 4096 * j);
#pragma unroll
    for (int i = 0; i < kFM; ++i) o.a[i] = *reinterpret_cast<const i32x4_t *>(smem + (xo ^ (32u * s)) + 4096 * i);
  };
  // One step on the current stage while the next one (of this tile or the
  // next) is fetched into the other: fetch issues it.
  auto step = [&](auto lora, auto fetch) __attribute__((always_inline)) {
    constexpr bool kLora = decltype(lora)::value;
    uint32_t ha[kHold], hb[kFN];   // scales of the products held back (sub-step 3)
#pragma unroll
    for (int i = 0; i < kHold; ++i) ha[i] = sc.a[kFM - kHold + i].y;
#pragma unroll
    for (int j = 0; j < kFN; ++j) hb[j] = sc.b[j].y;
    read(fa, 0);
    if constexpr (!kLora) {
#pragma unroll
      for (int i = 0; i < kFM; ++i) sc.a[i] = *reinterpret_cast<const uint2 *>(smem + so + 256 * i);
#pragma unroll
      for (int j = 0; j < kFN; ++j) sc.b[j] = *reinterpret_cast<const uint2 *>(smem + to + 256 * j);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kHold; ++i)
#pragma unroll
      for (int j = 0; j < kFN; ++j) {
        f32x16_t &c = acc[kFM - kHold + i][j];
        c = mul1<kBf16>(fb.a[kFM - kHold + i], fb.b[j], ha[i], hb[j], 3, c);
      }
    fetch(1);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!kLora) {
#pragma unroll
      for (int i = 0; i < kFM; ++i) sc.a[i] = make_uint2(sc.a[i].x >> (8 * lh), sc.a[i].y >> (8 * lh));
#pragma unroll
      for (int j = 0; j < kFN; ++j) sc.b[j] = make_uint2(sc.b[j].x >> (8 * lh), sc.b[j].y >> (8 * lh));
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      Ops<kFM, kFN> &cur = (s & 1) ? fb : fa;
      Ops<kFM, kFN> &nxt = (s & 1) ? fa : fb;
      mul<0, 1, kLora>(cur, sc, s, acc);
      __builtin_amdgcn_sched_barrier(0);
      if (s < 3) read(nxt, s + 1);
      mul<1, kFM - kHold, kLora>(cur, sc, s, acc);
      __builtin_amdgcn_sched_barrier(0);
      if (s < 3) mul<kFM - kHold, kFM, kLora>(cur, sc, s, acc);
      if (s == 0) fetch(2);
      __builtin_amdgcn_sched_barrier(0);
    }
    xo ^= kStX;
    wo ^= kStW;
    so ^= kStS;
    to ^= kStS;
    raw_barrier<wait_imm(0, 0)>();
  };

  int m0, n0;
  Tiles::place(args, tiles.next, kBM, kBN, m0, n0);
  uint32_t st = 0;
  dma(0, m0, n0, k0, 3);
  raw_barrier<wait_imm(0, 0)>();
  for (;;) {
    clear();
    tiles.next += tiles.step;
    const bool more = tiles.next < tiles.end;
    int m1 = 0, n1 = 0;
    if (more) Tiles::place(args, tiles.next, kBM, kBN, m1, n1);
    auto fetch = [&](int kt, int part) __attribute__((always_inline)) {
      if (part & 1) st ^= 1;
      if (kt + 1 < steps)
        dma(st, m0, n0, kt + 1, part);
      else if (more)
        dma(st, m1, n1, k0, part);
    };
    for (int kt = k0; kt < k1; ++kt) step(std::bool_constant<kBf16>(), [&](int part) __attribute__((always_inline)) { fetch(kt, part); });
    if (kPiped && last) {
      step(std::true_type(), [&](int part) __attribute__((always_inline)) { fetch(KT, part); });
      mul<kFM - kHold, kFM, true>(fb, sc, 3, acc);
    } else {
      mul<kFM - kHold, kFM, kBf16>(fb, sc, 3, acc);
      // The stage just consumed takes T and B; the other one is being filled.
      for (int j0 = 0; !kPiped && last && j0 < r; j0 += 64) {
        stage_narrow<kBM>(smem + (st ? 0 : kStX), args.T, r, m0, M, j0);
        stage_narrow<kBN>(smem + kOffW + (st ? 0 : kStW), args.B, r, n0, N, j0);
        __syncthreads();
        xo ^= kStX;
        wo ^= kStW;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          read(fa, s);
          mul<0, kFM, true>(fa, sc, s, acc);
        }
        xo ^= kStX;
        wo ^= kStW;
        __syncthreads();
      }
    }

    if constexpr (kSplit) {
      float4 *out = reinterpret_cast<float4 *>(args.part) +
                    ((static_cast<int64_t>(split) * args.trows * args.tcols + tile) * 8 + wave) * (kFM * kFN * 256) + lane;
#pragma unroll
      for (int i = 0; i < kFM; ++i)
#pragma unroll
        for (int j = 0; j < kFN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            out[((i * kFN + j) * 4 + q) * 64] = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                                            acc[i][j][4 * q + 3]);
      return;
    }

    // Accumulator layout: lane l holds row m = l % 32 of Y; element e is
    // column 8 (e / 4) + 4 (l / 32) + e % 4.  Each 32 rows go through the part
    // of the consumed stage that this wave's own next fetch fills, so that a
    // store instruction covers whole row segments (16 bytes of 32 rows each
    // would take twice the address cycles).
    constexpr int kChunks = 4 * kFN, kRowsOnce = 64 / kChunks;   // 16-byte chunks of the wave's columns
    uint8_t *part = smem + (st ? 0 : kStX) + wave * (kBM * 16);
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
#pragma unroll
      for (int j = 0; j < kFN; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = pack_bf16x2(acc[i][j][8 * q + 2 * e], acc[i][j][8 * q + 2 * e + 1]);
          swap_halves(p[0], p[2]);
          swap_halves(p[1], p[3]);
          const int c = 4 * j + 2 * q + lh;
          *reinterpret_cast<uint4 *>(part + 16 * (lr * kChunks + (c ^ (lr & (kChunks - 1))))) =
              make_uint4(p[0], p[1], p[2], p[3]);
        }
      __builtin_amdgcn_s_waitcnt(wait_imm(63, 0));
#pragma unroll
      for (int t = 0; t < 32 / kRowsOnce; ++t) {
        const int rr = t * kRowsOnce + lane / kChunks, c = lane % kChunks;
        const uint4 v = *reinterpret_cast<const uint4 *>(part + 16 * (rr * kChunks + (c ^ (rr & (kChunks - 1)))));
        const int m = m0 + 32 * (kFM * wm + i) + rr, n = n0 + 32 * kFN * wn + 8 * c;
        uint16_t *y = args.Y + static_cast<int64_t>(m) * N + n;
        if (m < M && n + 8 <= N) {
          *reinterpret_cast<uint4_any *>(y) = v;
        } else if (m < M) {
          const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < N) y[e] = static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1)));
        }
      }
      __builtin_amdgcn_s_waitcnt(wait_imm(63, 0));   // read before the next 32 rows, or the next fetch, write there
    }
    if (!more) return;
    m0 = m1;
    n0 = n1;
  }
}

// One workgroup: one wave's part of a tile, its splits' sums added in order.
template <int kFM, int kFN>
__global__ __launch_bounds__(kFM * kFN * 256) void k_mx4_join(const Mx4Args args) {
  const int lane = threadIdx.x & 63, part = threadIdx.x >> 6;     // part: fragment and quarter of its elements
  const int tile = blockIdx.x >> 3, wave = blockIdx.x & 7;
  const int64_t plane = static_cast<int64_t>(args.trows) * args.tcols * 8 * (kFM * kFN * 256);
  const float4 *p = reinterpret_cast<const float4 *>(args.part) + static_cast<int64_t>(blockIdx.x) * (kFM * kFN * 256) + threadIdx.x;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int z = 0; z < args.splits; ++z) {
    const float4 v = p[z * plane];
    t.x += v.x;
    t.y += v.y;
    t.z += v.z;
    t.w += v.w;
  }
  int m0, n0;
  Tiles::place(args, tile, 64 * kFM, 128 * kFN, m0, n0);
  const int f = part >> 2, q = part & 3;
  const int m = m0 + 32 * (kFM * (wave >> 2) + f / kFN) + (lane & 31);
  const int n = n0 + 32 * (kFN * (wave & 3) + f % kFN) + 8 * q + 4 * (lane >> 5);
  if (m >= args.M) return;
  uint16_t *y = args.Y + static_cast<int64_t>(m) * args.N + n;
  const uint32_t a = pack_bf16x2(t.x, t.y), b = pack_bf16x2(t.z, t.w);
  typedef uint2 __attribute__((aligned(2))) uint2_any;
  if (n + 4 <= args.N) {
    *reinterpret_cast<uint2_any *>(y) = make_uint2(a, b);
  } else {
    const uint32_t h[2] = {a, b};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < args.N) y[e] = static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1)));
  }
}

namespace {

int64_t small_tiles(int64_t M, int64_t N) { return (M + 127) / 128 * ((N + 127) / 128); }

// Parts of the contraction for few small tiles, four steps or more each.  A
// step of a lone workgroup waits for its fetch, some 0.7 us; partial tiles and
// join cost about 20 such steps.  Whole and split, with the join:
//   128 x 4096 x 11008   32.3   16.3 us   (10 parts: 38 steps saved)
//   512 x 4096 x 11008   32.8   28.2      (3 parts: 28)
//   512 x 4096 x 6144    19.2   21.2      (3 parts: 16)
//   256 x 11008 x 8192   25.4   28.0      (2 parts: 16)
int splits_of(int64_t M, int64_t N, int64_t K) {
  const int64_t KT = mx4_slabs(K);
  const int64_t z = std::max<int64_t>(1, std::min(KT / 4, 384 / small_tiles(M, N)));
  return KT - KT / z >= 20 ? static_cast<int>(z) : 1;
}

template <int kFM, int kFN>
hipError_t launch_tiles(Mx4Args a, int per_cu, hipStream_t s) {
  a.trows = (a.M + 64 * kFM - 1) / (64 * kFM);
  a.tcols = (a.N + 128 * kFN - 1) / (128 * kFN);
  const int64_t tiles = static_cast<int64_t>(a.trows) * a.tcols;
  const dim3 block(kMxMmThreads);
  if constexpr (kFM == 2) {
    if (a.splits > 1) {
      const dim3 grid(static_cast<uint32_t>(tiles * a.splits));
      if (a.r == 64)
        hipLaunchKernelGGL((k_mx4_matmul<kFM, kFN, true, true>), grid, block, 0, s, a);
      else
        hipLaunchKernelGGL((k_mx4_matmul<kFM, kFN, false, true>), grid, block, 0, s, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL((k_mx4_join<kFM, kFN>), dim3(static_cast<uint32_t>(tiles * 8)), dim3(kFM * kFN * 256), 0, s, a);
      return hipGetLastError();
    }
  }
  const dim3 grid(static_cast<uint32_t>(std::min<int64_t>(tiles, kCUs * per_cu)));
  if (a.r == 64)
    hipLaunchKernelGGL((k_mx4_matmul<kFM, kFN, true, false>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_mx4_matmul<kFM, kFN, false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Parts of the contraction of dX, in steps of 64 columns.
int dx_splits_of(int64_t M, int64_t N, int64_t K) {
  const int64_t KT = N / 64;
  return static_cast<int>(std::max<int64_t>(1, std::min(KT / 4, 384 / small_tiles(M, K))));
}

}  // namespace

// While the small tiles all run at once: k_matmul_pre gives a large tile a whole
// contraction, 1.3 to 1.45 us a step of 64 columns however few tiles there are.  Both with
// the weight's decoding (and transposition here), us:
//   128 x 4096 from 11008   57   233        1024 x 4096 from 4096   71   95
//   707 x 256 from 3264     18    75        2048 x 4096 from 4096   91  105
//   1470 x 960 from 1408    22    40        2048 x 4096 from 1024   39   37
// Under 4 steps there is nothing to win (300 x 4096 from 192: 17.5 and 17.4).
// Offsets of a tile's rows are 32-bit.
bool mx4_dx_small_ok(int64_t M, int64_t N, int64_t K) {
  return N >= 256 && N <= (int64_t{1} << 20) && small_tiles(M, K) <= 2 * kCUs;
}

size_t mx4_dx_small_ws_bytes(int64_t M, int64_t N, int64_t K) {
  return mx4_dx_small_ok(M, N, K) ? static_cast<size_t>(dx_splits_of(M, N, K)) * small_tiles(M, K) * 128 * 128 * sizeof(float) : 0;
}

hipError_t launch_mx4_dx_small(const uint16_t *dY, const uint16_t *Wt, const uint16_t *G, const uint16_t *At, int M, int N,
                               int K, int r, uint16_t *dX, void *ws, hipStream_t s) {
  Mx4Args a{};
  a.xc = reinterpret_cast<const uint8_t *>(dY);
  a.wc = reinterpret_cast<const uint8_t *>(Wt);
  a.T = G;
  a.B = At;
  a.Y = dX;
  a.M = M;
  a.N = K;
  a.r = r;
  a.KT = N / 64;
  a.part = static_cast<float *>(ws);
  a.splits = dx_splits_of(M, N, K);
  a.trows = (M + 127) / 128;
  a.tcols = (K + 127) / 128;
  const int tiles = a.trows * a.tcols;
  const dim3 grid(static_cast<uint32_t>(tiles * a.splits)), block(kMxMmThreads);
  if (r == 64)
    hipLaunchKernelGGL((k_mx4_matmul<2, 1, true, true, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_mx4_matmul<2, 1, false, true, true>), grid, block, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_mx4_join<2, 1>), dim3(static_cast<uint32_t>(tiles * 8)), dim3(512), 0, s, a);
  return hipGetLastError();
}

size_t mx4_split_ws_bytes(int64_t M, int64_t N, int64_t K) {
  const int z = splits_of(M, N, K);
  return z > 1 ? static_cast<size_t>(z) * small_tiles(M, N) * 128 * 128 * sizeof(float) : 0;
}

hipError_t launch_mx4_matmul(const Mx4View &X, const Mx4View &W, const uint16_t *T, const uint16_t *B, int r, uint16_t *Y,
                             void *ws, hipStream_t s) {
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
  a.part = static_cast<float *>(ws);
  a.splits = ws ? splits_of(X.rows, W.rows, X.cols) : 1;
  // Small tiles while all of them run at once, two a compute unit (2048 x 4096
  // x 4096: 23.7 us, large 30.1); beyond, the large ones, which read half as
  // much (2048 x 5120 x 11008: 71.6 us, small 78.8; 8192 x 11008 x 4096: 206,
  // small 243).  A single small tile row would be half a large one (100 x 131072
  // x 4096: 64.9 us, large 72.7).
  return X.rows > 128 && small_tiles(X.rows, W.rows) > 2 * kCUs ? launch_tiles<4, 2>(a, 1, s) : launch_tiles<2, 1>(a, 2, s);
}

}  // namespace qlora
