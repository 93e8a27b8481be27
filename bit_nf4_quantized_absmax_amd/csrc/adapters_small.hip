// The linear layer with many adapters for up to 64 tokens (decoding):
//     Y_m = X_m deq(W)^T + T_m B_a^T,   T_m = bf16(scale_a X_m A_a^T),   a = index[m]
// Bound by the bytes of the packed weight and of the adapters in use, then by
// latency: two launches.  64 tokens x 11008 x 4096 with 64 adapters of rank 16 take
// 31 us (56 MB, 11 us at the rate of a copy; 23 of k_ad_stream and 11 of k_ad_epi in a
// trace), with one adapter 27; one token x 4096 x 4096 with rank 64 takes 9 + 4.
//
//  * k_ad_stream: one workgroup per CU, persistent, over equal ranges of
//    units (kPT x 64 weight rows by 256 columns).  A unit's packed codes, block
//    codes, group scales and X columns are DMA'd global -> LDS two units ahead; a
//    wave multiplies 16 rows by one 64-wide block: codes go through a byte ->
//    bf16x2 table of the levels into 16 x 16 x 32 products, each block's scaled by
//    its constant in fp32 (the weight is bf16(level) times the constant, as in the
//    framework's other decoding kernels).  Sums of a row tile go, in fp32, to a slot
//    for each workgroup that had a part of it.  K is any multiple of 64: columns past
//    it are zeros of X.  16 waves a workgroup: a wave waits for one table read after
//    another, so four share a SIMD (64 x 11008 x 4096, both kernels: 43 us with 8 waves of
//    32 rows, 37 with 16).
//  * Beside its first DMAs every wave takes its share of the products X A^T, 16
//    adapter rows by 512 columns each; every 16th token of an adapter stands for
//    itself and the next 15, which a ballot over the indices finds.
//  * k_ad_epi: 16 weight rows a workgroup; adds the slots in workgroup order, forms T
//    from its partial sums and adds each token's product with its own adapter: the
//    adapters in use go to the waves in turn, and a token takes the product of
//    its own only.  One rounding to bf16.
#include <algorithm>

#include "common.h"
#include "launch.h"
#include "lds_dma.h"
#include "tile.h"

namespace qlora {

__constant__ uint32_t cAdQ4Level[3 * 16] = {QLORA_Q4_LEVEL_BITS};
__constant__ uint32_t cAdT8Level[256] = {QLORA_T8_LEVEL_BITS};
__device__ const uint4 gAdZero[1] = {{0, 0, 0, 0}};   // what a DMA past a row reads

namespace {

constexpr int kThreads = 1024;               // of k_ad_stream
constexpr int kEpiThreads = 512;
constexpr int kRows = 64;                    // weight rows of a tile
constexpr int kUnitK = 256;
constexpr int kTileW = kRows * 128;          // packed bytes of a tile and unit
constexpr int kTileStage = kTileW + 1024;    // + 8 bytes of block codes and two group scales a row
constexpr int kLutCopies = 32;
constexpr int kSlice = 512;                  // columns of a partial sum of T
constexpr int kGridMax = 256;

// Row tiles of a unit where there are many units (a round's fixed cost counts): as
// the LDS allows; one tile where that leaves a workgroup few (their even share counts).
constexpr int many_tiles(int kmb) { return kmb == 1 ? 3 : 2; }
// Stages of X (3: two units ahead, 2: one).
template <int kMB>
constexpr int x_stages() { return kMB == 4 ? 2 : 3; }

__device__ __forceinline__ void dma4_far(const void *src, uint32_t dst) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "{m0}"(dst) : "memory");
}

// Swizzled places: weight rows (128 bytes, 8 chunks) and X rows (512 bytes, 32 chunks).
__device__ __forceinline__ int wpos(int row, int chunk) { return row * 128 + 16 * (chunk ^ ((row >> 1) & 7)); }
__device__ __forceinline__ int xpos(int row, int chunk) { return row * 512 + 16 * (chunk ^ (row & 15)); }

// First unit of workgroup w of G over U units, and the workgroup of a unit (N K < 2^31: U <= 2^20; G <= 256).
__device__ __forceinline__ int first_unit(int w, int G, int U) {
  return static_cast<int>(static_cast<uint32_t>(w * U) / static_cast<uint32_t>(G));
}
__device__ __forceinline__ int workgroup_of(int u, int G, int U) {
  int w = static_cast<int>(static_cast<uint32_t>(u * G) / static_cast<uint32_t>(U));
  while (w + 1 < G && first_unit(w + 1, G, U) <= u) ++w;
  while (w > 0 && first_unit(w, G, U) > u) --w;
  return w;
}

__device__ __forceinline__ int adapter_of(const int64_t *index, int m, int n) {
  const int64_t a = index[m];
  return a >= 0 && a < n ? static_cast<int>(a) : -1;
}

// Slot of tile t of group `group` summed by workgroup w: groups and workgroups rise together, so group + w is its own.
template <int kMB, int kPT>
__device__ __forceinline__ float *slot(float *slots, int group, int t, int w) {
  constexpr int kPiece = 4 * kMB * 64 * 4;
  return slots + (static_cast<int64_t>(group + w) * kPT + t) * kPiece;
}

struct StreamArgs {
  const uint16_t *X;
  NF4View w;
  AdapterSet ad;
  float *P;        // [slices][M][r]
  float *slots;
  int M, KT, groups;
};

// One wave's share of the partial sums of T: items (token, 16 adapter rows, slice), of
// which every 16th token of an adapter stands for itself and the next 15.  mine: the
// adapter of token `lane`, -1: none.
__device__ __forceinline__ void down_items(const StreamArgs &a, int mine, int item0, int step) {
  const int lane = threadIdx.x & 63, nl = lane & 15, g = lane >> 4;
  const int M = a.M, K = a.w.K, r = a.ad.r;
  const int jts = (r + 15) >> 4, slices = (K + kSlice - 1) / kSlice;
  for (int it = item0; it < M * jts * slices; it += step) {
    const int m0 = it % M, jt = it / M % jts, sl = it / M / jts;
    const int ad = __builtin_amdgcn_readlane(mine, m0);
    const uint64_t mask = __ballot(mine == ad);
    const int cnt = __popcll(mask), t0 = __popcll(mask & ((uint64_t{1} << m0) - 1));
    if (ad < 0 || (t0 & 15) != 0) continue;
    // token number t0 + nl of the adapter (0 past the last: its column is not stored)
    const int rank = __popcll(mask & ((uint64_t{1} << lane) - 1)) - t0;
    const int sent = __builtin_amdgcn_ds_permute(4 * (mine == ad && rank >= 0 && rank < 16 ? rank : 63), lane);
    const int tok = __builtin_amdgcn_ds_bpermute(4 * nl, sent);
    const int j = 16 * jt + nl;
    const uint16_t *arow = a.ad.A + (static_cast<int64_t>(ad) * r + min(j, r - 1)) * K;
    const int k0 = sl * kSlice, steps = min(kSlice, K - k0) >> 5;   // K % 64 == 0
    float *P = a.P + static_cast<int64_t>(sl) * M * r;
    const uint16_t *xrow = a.X + static_cast<int64_t>(tok) * K;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s0 = 0; s0 < steps; s0 += 8) {
      bf16x8_t av[8], xv[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = k0 + 32 * min(s0 + u, steps - 1) + 8 * g;
        av[u] = *reinterpret_cast<const bf16x8_t *>(arow + k);
        xv[u] = *reinterpret_cast<const bf16x8_t *>(xrow + k);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (s0 + u < steps) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[u], xv[u], acc, 0, 0, 0);
    }
    // lane: token nl, adapter rows 16 jt + 4 g + e
    if (t0 + nl < cnt && 16 * jt + 4 * g < r) *reinterpret_cast<f32x4_t *>(P + static_cast<int64_t>(tok) * r + 16 * jt + 4 * g) = acc;
  }
}

}  // namespace

template <int kMB, int kPT>
__global__ __launch_bounds__(kThreads) void k_ad_stream(const StreamArgs a) {
  constexpr int kXS = x_stages<kMB>(), kWS = 3;
  constexpr int kXStage = kMB * 16 * 512;
  constexpr int kWStage = kPT * kTileStage;
  constexpr int kWaves = kThreads / 64;
  // DMA instructions of a unit, to the waves in turn: 8 kPT of codes and 4 kPT of block
  // codes and group scales (W), 8 kMB of X.  At the end of a unit all but the newest
  // may be in flight: with three X stages W and X of the unit after next, with two (X
  // is issued before W) only its W.
  constexpr int kDmaW = 12 * kPT, kDmaX = 8 * kMB;
  __shared__ __attribute__((aligned(16))) uint8_t sX[kXS * kXStage];
  __shared__ __attribute__((aligned(16))) uint8_t sW[kWS * kWStage];
  __shared__ uint32_t sLut[256 * kLutCopies];
  __shared__ float sT8[256];
  const int G = gridDim.x, w = blockIdx.x;
  const int U = a.groups * a.KT;
  const int u0 = first_unit(w, G, U), u1 = first_unit(w + 1, G, U);
  if (u0 >= u1) return;                      // (the grid never exceeds the unit count)
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rq = wave & 3, kq = wave >> 2;       // 16 rows of a tile, block of a unit
  const int nl = lane & 15, g = lane >> 4;
  const int M = a.M, N = a.w.N, K = a.w.K, KB = K >> 6;
  const float mean = a.w.mean[0];
  // The index and the levels are waited for together and before the first DMA is issued:
  // a wait behind the DMAs would be for them too.
  const int64_t named = lane < M ? a.ad.index[lane] : -1;
  {
    // Wave w writes the bytes whose low half is w, a copy a lane: uniform loads.
    static_assert(kWaves == 16 && kLutCopies == 32, "a wave a level, two bytes at a time");
    const uint32_t *level = cAdQ4Level + 16 * a.w.qtype;
    const float lo = u2f(level[wave]);
    uint32_t *dst = sLut + wave * kLutCopies + (lane & 31);
#pragma unroll
    for (int j = 0; j < 16; j += 2)
      dst[16 * kLutCopies * (j + (lane >> 5))] = pack_bf16x2(lo, u2f(lane < 32 ? level[j] : level[j + 1]));
  }

  const int mine = named >= 0 && named < a.ad.n ? static_cast<int>(named) : -1;

  const uint32_t xbase = lds_addr(sX), wbase = lds_addr(sW);
  // X: instruction i fills rows 2 i and 2 i + 1 of a stage, 32 chunks each; rows past M
  // repeat the last, chunks past K are zeros.
  constexpr int kMineX = (kDmaX + kWaves - 1) / kWaves;
  const uint16_t *xsrc[kMineX];
  int xk[kMineX];
#pragma unroll
  for (int j = 0; j < kMineX; ++j) {
    const int row = 2 * (wave + kWaves * j) + (lane >> 5);
    xk[j] = 8 * ((lane & 31) ^ (row & 15));
    xsrc[j] = a.X + static_cast<int64_t>(min(row, M - 1)) * K + xk[j];
  }
  auto dma_x = [&](int q, int kt) __attribute__((always_inline)) {
    const uint32_t dst = xbase + (q % kXS) * kXStage;
#pragma unroll
    for (int j = 0; j < kMineX; ++j) {
      const int i = wave + kWaves * j;
      if (i >= kDmaX) break;                     // uniform
      const void *src = kUnitK * kt + xk[j] < K ? static_cast<const void *>(xsrc[j] + kUnitK * kt) : gAdZero;
      dma16(src, __builtin_amdgcn_readfirstlane(dst + i * 1024));
    }
  };
  // W: instruction 8 t + i fills rows 8 i .. 8 i + 7 of tile t, 8 kPT + 4 t + part the rows'
  // words of a part: 0, 1 the aligned words that hold the row's block codes 4 kt .. + 3,
  // 2, 3 the scales of the first's and last's groups.  Chunks past K (they meet
  // zeros) and rows past N (never stored) repeat the last.
  const int64_t codes = static_cast<int64_t>(N) * KB;
  auto dma_w = [&](int q, int group, int kt) __attribute__((always_inline)) {
    const uint32_t dst = wbase + (q % kWS) * kWStage;
#pragma unroll
    for (int i = wave; i < kDmaW; i += kWaves) {
      if (i < 8 * kPT) {
        const int t = i >> 3, row = 8 * (i & 7) + (lane >> 3);
        const int n = min(kRows * (kPT * group + t) + row, N - 1);
        const int byte = min(128 * kt + 16 * ((lane & 7) ^ ((row >> 1) & 7)), (K >> 1) - 16);
        dma16(a.w.packed + static_cast<int64_t>(n) * (K >> 1) + byte,
              __builtin_amdgcn_readfirstlane(dst + t * kTileStage + (i & 7) * 1024));
      } else {
        const int t = (i - 8 * kPT) >> 2, part = i & 3;
        const int n = min(kRows * (kPT * group + t) + lane, N - 1);
        const int64_t cb = static_cast<int64_t>(n) * KB + 4 * kt;
        const void *src;
        if (part < 2)
          src = a.w.code8 + min((cb & ~int64_t{3}) + 4 * part, (codes - 1) & ~int64_t{3});
        else
          src = a.w.c2 + (min(cb + (part == 2 ? 0 : 3), codes - 1) >> 8);
        dma4_far(src, __builtin_amdgcn_readfirstlane(dst + t * kTileStage + kTileW + part * 256));
      }
    }
  };
  // This wave's instructions among those.
  const int ahead = (kDmaW - wave + kWaves - 1) / kWaves + (kXS == 3 ? (kDmaX - wave + kWaves - 1) / kWaves : 0);
  constexpr int kAheadMax = (kDmaW + kWaves - 1) / kWaves + (kXS == 3 ? kMineX : 0);
  static_assert(kAheadMax <= 6, "the cases below");
  auto unit_end = [&]() __attribute__((always_inline)) {
    switch (ahead) {                             // uniform
      case 0: raw_barrier<wait_imm(0, 0)>(); break;
      case 1: raw_barrier<wait_imm(1, 0)>(); break;
      case 2: raw_barrier<wait_imm(2, 0)>(); break;
      case 3: raw_barrier<wait_imm(3, 0)>(); break;
      case 4: raw_barrier<wait_imm(4, 0)>(); break;
      case 5: raw_barrier<wait_imm(5, 0)>(); break;
      default: raw_barrier<wait_imm(6, 0)>(); break;
    }
  };

  const int nq = u1 - u0;
  // Places in the range: of the products, of the weights' DMA, of X's (past the range both repeat the last unit).
  struct Pos {
    int group, kt;
  };
  auto next = [&](Pos &p) __attribute__((always_inline)) {
    if (++p.kt == a.KT) {
      p.kt = 0;
      ++p.group;
    }
  };
  Pos pc{u0 / a.KT, u0 % a.KT}, pw = pc, px = pc;
  int qw = 0, qx = 0;
  auto issue_w = [&]() __attribute__((always_inline)) {
    dma_w(qw, pw.group, pw.kt);
    if (++qw < nq) next(pw);
  };
  auto issue_x = [&]() __attribute__((always_inline)) {
    dma_x(qx, px.kt);
    if (++qx < nq) next(px);
  };
  if (wave < 4) dma4_far(cAdT8Level + tid, __builtin_amdgcn_readfirstlane(lds_addr(sT8) + 256 * wave));
  if constexpr (kXS == 3) {
    issue_w();
    issue_x();
    issue_w();
    issue_x();
  } else {
    issue_x();
    issue_w();
    issue_w();
  }
  down_items(a, mine, wave * G + w, G * kWaves);
  unit_end();

  f32x4_t acc[kPT][kMB];
#pragma unroll
  for (int t = 0; t < kPT; ++t)
#pragma unroll
    for (int mb = 0; mb < kMB; ++mb) acc[t][mb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint32_t lutl = static_cast<uint32_t>(lane & 31);

  for (int q = 0; q < nq; ++q) {
    if constexpr (kXS == 3) {
      issue_w();                                 // weights of unit q + 2, X of q + 2 or q + 1
      issue_x();
    } else {
      issue_x();
      issue_w();
    }
    const int group = pc.group, kt = pc.kt;
    next(pc);
    const uint8_t *xs = sX + (q % kXS) * kXStage;
    const uint8_t *ws0 = sW + (q % kWS) * kWStage;
    bf16x8_t xa[kMB][2];
#pragma unroll
    for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
        xa[mb][tt] = *reinterpret_cast<const bf16x8_t *>(xs + xpos(16 * mb + nl, 8 * kq + 2 * g + tt));
#pragma unroll
    for (int t = 0; t < kPT; ++t) {
      const uint8_t *ws = ws0 + t * kTileStage;
      const int row = 16 * rq + nl;
      const int n = min(kRows * (kPT * group + t) + row, N - 1);
      const uint32_t cb = static_cast<uint32_t>(n) * static_cast<uint32_t>(KB) + 4 * kt;   // below 2^25
      const uint32_t at = (cb & 3) + kq;         // byte of the row's two words
      const int code = ws[kTileW + 256 * (at >> 2) + 4 * row + (at & 3)];
      const int far = ((cb + kq) >> 8) != (cb >> 8) ? 1 : 0;
      const float c2 = *reinterpret_cast<const float *>(ws + kTileW + 512 + 256 * far + 4 * row);
      const uint2 pk = *reinterpret_cast<const uint2 *>(ws + wpos(row, 2 * kq + (g >> 1)) + 8 * (g & 1));
      const float chat = decode_absmax(sT8[code], c2, mean);
      const uint32_t words[2] = {pk.x, pk.y};
      bf16x8_t wop[2];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = sLut[((words[tt] >> (8 * i)) & 0xffu) * kLutCopies + lutl];
        wop[tt] = __builtin_bit_cast(bf16x8_t, o);
      }
#pragma unroll
      for (int mb = 0; mb < kMB; ++mb) {
        f32x4_t part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[mb][0], wop[0], f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[mb][1], wop[1], part, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][mb][e] = __builtin_fmaf(chat, part[e], acc[t][mb][e]);
      }
    }
    unit_end();

    if (kt == a.KT - 1 || q == nq - 1) {
      // A tile's four block quarters are added ((0 + 2) + (1 + 3)) in this unit's X
      // stage, which is consumed and not filled again before the next unit.
      f32x4_t *red = reinterpret_cast<f32x4_t *>(sX + (q % kXS) * kXStage);
      auto at = [&](int s, int mb) -> f32x4_t & { return red[((s * 4 + rq) * kMB + mb) * 64 + lane]; };
#pragma unroll
      for (int t = 0; t < kPT; ++t) {
#pragma unroll
        for (int mb = 0; mb < kMB; ++mb)
          if (kq >= 2) at(kq - 2, mb) = acc[t][mb];
        raw_barrier<wait_imm(63, 0)>();
#pragma unroll
        for (int mb = 0; mb < kMB; ++mb)
          if (kq < 2) {
            acc[t][mb] += at(kq, mb);
            if (kq == 1) at(1, mb) = acc[t][mb];
          }
        raw_barrier<wait_imm(63, 0)>();
        if (kq == 0) {
          f32x4_t *dst = reinterpret_cast<f32x4_t *>(slot<kMB, kPT>(a.slots, group, t, w));
#pragma unroll
          for (int mb = 0; mb < kMB; ++mb) dst[(rq * kMB + mb) * 64 + lane] = acc[t][mb] + at(1, mb);
        }
        raw_barrier<wait_imm(63, 0)>();          // red is used again by the next tile
#pragma unroll
        for (int mb = 0; mb < kMB; ++mb) acc[t][mb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
  }
  raw_barrier<wait_imm(0, 0)>();                 // the repeated DMAs past the range
}

// Workgroup: 16 weight rows, all tokens, 8 waves, which take the adapters in use in
// turn.  An adapter's tokens are the rows of its own products, 16 at a time (lane:
// weight row l % 16, token 4 (l / 16) + e of them), so every token's sum is written
// by one wave.  kH: 32-column parts of B that are fetched at once (1: r <= 32).  The
// first adapters' rows of B and the partial sums of T are all asked for before the first
// is used.  Registers for three workgroups a compute unit: 688 of them (N = 11008) are one
// round then, where two make a second (both kernels 31.6 us against 36.7; rank 64, with
// two adapters' rows in flight instead of four, 50 against 54).
template <int kMB, int kPT, int kH>
__global__ __launch_bounds__(kEpiThreads, 6) void k_ad_epi(const StreamArgs a, int G, uint16_t *__restrict__ Y, uint16_t *__restrict__ T) {
  constexpr int kWaves = kEpiThreads / 64;
  constexpr int kAtOnce = kMB == 1 || kH == 2 ? 2 : 4;            // adapters whose rows of B are in flight
  constexpr int kSeg = 4;                              // slots likewise
  __shared__ __attribute__((aligned(16))) uint16_t sT[64 * 136];   // T, rows of r + 8
  __shared__ float sL[64][17];                         // the adapters' term
  __shared__ int sAd[64], sRank[64], sList[64], sTok[kWaves][64], sCount[kAdMax], sUsed;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, g = lane >> 4;
  const int M = a.M, N = a.w.N, r = a.ad.r, pitch = r + 8;
  const int n0 = 16 * blockIdx.x, n = min(n0 + nl, N - 1);
  const int tile = blockIdx.x >> 2, group = tile / kPT, t = tile % kPT;
  const int mine = lane < M ? adapter_of(a.ad.index, lane, a.ad.n) : -1;
  const int slices = (a.w.K + kSlice - 1) / kSlice;
  const int U = a.groups * a.KT;
  const int wf = workgroup_of(group * a.KT, G, U), wl = workgroup_of(group * a.KT + a.KT - 1, G, U);
  // A token's number among those of its adapter (in any order: it is the row of a
  // product that its sum comes from); the first of each stands for it.
  if (wave == 0) {
    sAd[lane] = mine;
    int rank = 0;
    if (mine >= 0) {
      sCount[mine] = 0;
      rank = atomicAdd(&sCount[mine], 1);
    }
    sRank[lane] = rank;
    const uint64_t firsts = __ballot(mine >= 0 && rank == 0);
    if (mine >= 0 && rank == 0) sList[__popcll(firsts & ((uint64_t{1} << lane) - 1))] = mine;
    if (lane == 0) sUsed = __popcll(firsts);
  }
  __syncthreads();
  const int rank = sRank[lane], used = sUsed;
  const int list = sList[lane];                        // lane i: the i-th adapter in use (i < used)
  bf16x8_t bop[kAtOnce][kH];
  auto fetch = [&](int i0, int j0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int ad = __builtin_amdgcn_readlane(list, min(i0 + kWaves * u, used - 1));
      const uint16_t *brow = a.ad.B + (static_cast<int64_t>(ad) * N + n) * r;
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const int j = j0 + 32 * h + 8 * g;
        bop[u][h] = *reinterpret_cast<const bf16x8_t *>(brow + (j < r ? j : 0));
      }
    }
  };
  if (wave < used) fetch(wave, 0);
  // T from its partial sums, in slice order.
  for (int i = tid; i < M * (r >> 2); i += kEpiThreads) {
    const int m = i / (r >> 2), j = 4 * (i % (r >> 2));
    const int x = sAd[m];
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    float s = 0.f;
    if (x >= 0) {
      s = a.ad.scale[x];
      const float *p = a.P + static_cast<int64_t>(m) * r + j;
      for (int c0 = 0; c0 < slices; c0 += 8) {
        f32x4_t q[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) q[c] = *reinterpret_cast<const f32x4_t *>(p + static_cast<int64_t>(min(c0 + c, slices - 1)) * M * r);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c0 + c < slices) v += q[c];
      }
    }
    const uint2 b = make_uint2(pack_bf16x2(s * v[0], s * v[1]), pack_bf16x2(s * v[2], s * v[3]));
    *reinterpret_cast<uint2 *>(sT + m * pitch + j) = b;
    if (blockIdx.x == 0) *reinterpret_cast<uint2 *>(T + static_cast<int64_t>(m) * r + j) = b;
  }
  // not earlier, for the registers' sake
  f32x4_t seg[kSeg];
  if (wave < kMB) {
#pragma unroll
    for (int i = 0; i < kSeg; ++i)
      seg[i] = reinterpret_cast<const f32x4_t *>(slot<kMB, kPT>(a.slots, group, t, min(wf + i, wl)))[((blockIdx.x & 3) * kMB + wave) * 64 + lane];
  }
  __syncthreads();
  for (int i0 = wave; i0 < used; i0 += kWaves * kAtOnce) {
    if (i0 != wave) fetch(i0, 0);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (i0 + kWaves * u >= used) break;              // uniform
      const int ad = __builtin_amdgcn_readlane(list, i0 + kWaves * u);
      const int cnt = __popcll(__ballot(mine == ad));
      if (mine == ad) sTok[wave][rank] = lane;
      for (int t0 = 0; t0 < cnt; t0 += 16) {
        const uint16_t *trow = sT + sTok[wave][min(t0 + nl, cnt - 1)] * pitch;
        f32x4_t part = {0.f, 0.f, 0.f, 0.f};
        for (int j0 = 0; j0 < r; j0 += 32 * kH) {
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            const int j = j0 + 32 * h + 8 * g;
            const bool ok = j < r;                     // r % 8 == 0
            bf16x8_t top = *reinterpret_cast<const bf16x8_t *>(trow + (ok ? j : 0));
            bf16x8_t bv = bop[u][h];
            if (j0 > 0) bv = *reinterpret_cast<const bf16x8_t *>(a.ad.B + (static_cast<int64_t>(ad) * N + n) * r + (ok ? j : 0));
            if (!ok) top = bv = bf16x8_t{};
            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(top, bv, part, 0, 0, 0);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t0 + 4 * g + e < cnt) sL[sTok[wave][t0 + 4 * g + e]][nl] = part[e];
      }
    }
  }
  __syncthreads();
  if (wave < kMB) {
    f32x4_t v = seg[0];
#pragma unroll
    for (int i = 1; i < kSeg; ++i)
      if (wf + i <= wl) v += seg[i];
    for (int w = wf + kSeg; w <= wl; ++w)
      v += reinterpret_cast<const f32x4_t *>(slot<kMB, kPT>(a.slots, group, t, w))[((blockIdx.x & 3) * kMB + wave) * 64 + lane];
    if (n0 + nl < N)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = 16 * wave + 4 * g + e;
        if (m < M) Y[static_cast<int64_t>(m) * N + n0 + nl] = f32_to_bf16(sAd[m] >= 0 ? v[e] + sL[m][nl] : v[e]);
      }
  }
}

// ---------------------------------------------------------------------------
namespace {

// Compute units of the current device, looked up once per device.
int compute_units() {
  static int known[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  if (known[dev] == 0) {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1) cus = 1;
    known[dev] = std::min(cus, kGridMax);
  }
  return known[dev];
}

int64_t row_tiles(int N) { return (static_cast<int64_t>(N) + kRows - 1) / kRows; }

// Tiles of a unit: one where a workgroup has fewer than kFew units of many.
constexpr int kFew = 4;
int unit_tiles(int M, int N, int K) {
  const int pt = many_tiles((M + 15) / 16);
  const int64_t units = (row_tiles(N) + pt - 1) / pt * ((K + kUnitK - 1) / kUnitK);
  return units < static_cast<int64_t>(kFew) * kGridMax ? 1 : pt;
}

size_t slot_bytes(int M, int N) {   // for either cut
  const int kmb = (M + 15) / 16, pt = many_tiles(kmb);
  const int64_t pieces = std::max((row_tiles(N) + pt - 1) / pt * pt + static_cast<int64_t>(kGridMax) * pt, row_tiles(N) + kGridMax);
  return static_cast<size_t>(pieces) * (4 * kmb * 64 * 4) * sizeof(float);
}

template <int kMB, int kPT>
hipError_t launch_cut(StreamArgs a, uint16_t *T, uint16_t *Y, hipStream_t s) {
  a.groups = static_cast<int>((row_tiles(a.w.N) + kPT - 1) / kPT);
  const int64_t units = static_cast<int64_t>(a.groups) * a.KT;
  const int grid = static_cast<int>(std::min<int64_t>(compute_units(), units));
  hipLaunchKernelGGL((k_ad_stream<kMB, kPT>), dim3(grid), dim3(kThreads), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 epi((a.w.N + 15) / 16);
  if (a.ad.r <= 32)
    hipLaunchKernelGGL((k_ad_epi<kMB, kPT, 1>), epi, dim3(kEpiThreads), 0, s, a, grid, Y, T);
  else
    hipLaunchKernelGGL((k_ad_epi<kMB, kPT, 2>), epi, dim3(kEpiThreads), 0, s, a, grid, Y, T);
  return hipGetLastError();
}

template <int kMB>
hipError_t launch_small(const StreamArgs &a, uint16_t *T, uint16_t *Y, hipStream_t s) {
  if (unit_tiles(a.M, a.w.N, a.w.K) == 1) return launch_cut<kMB, 1>(a, T, Y, s);
  return launch_cut<kMB, many_tiles(kMB)>(a, T, Y, s);
}

}  // namespace

size_t ad_small_ws_bytes(int M, int N, int K, int r) {
  const size_t p = static_cast<size_t>((K + kSlice - 1) / kSlice) * M * r * sizeof(float);
  return (p + 255) / 256 * 256 + slot_bytes(M, N);
}

hipError_t launch_ad_small(const uint16_t *X, int M, const NF4View &w, const AdapterSet &ad, uint16_t *T, uint16_t *Y, void *ws,
                           hipStream_t s) {
  const size_t p = static_cast<size_t>((w.K + kSlice - 1) / kSlice) * M * ad.r * sizeof(float);
  StreamArgs a{X, w, ad, static_cast<float *>(ws), reinterpret_cast<float *>(static_cast<char *>(ws) + (p + 255) / 256 * 256), M,
               (w.K + kUnitK - 1) / kUnitK, 0};
  switch ((M + 15) / 16) {
    case 1: return launch_small<1>(a, T, Y, s);
    case 2: return launch_small<2>(a, T, Y, s);
    case 3: return launch_small<3>(a, T, Y, s);
    default: return launch_small<4>(a, T, Y, s);
  }
}

}  // namespace qlora
