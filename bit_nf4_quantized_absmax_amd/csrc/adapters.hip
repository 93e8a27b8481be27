// Many LoRA adapters beside one frozen projection (gfx950): every token names
// the adapter of its request.
//     T_m  = s_a X_m A_a^T              Y_m  = X_m deq(W)^T + T_m B_a^T
//     G_m  = s_a dY_m B_a               dX_m = dY_m deq(W) + G_m A_a
//     dA_a = sum_m G_m^T X_m            dB_a = sum_m dY_m^T T_m   (m of adapter a)
// with a = index[m], A [n, r, K], B [n, N, r].  A token whose index is outside
// [0, n) has no adapter.
//
// Here for more than kAdSmall tokens, and for every backward pass (fewer tokens
// forward: adapters_small.hip).  The tokens are sorted by adapter once (k_ad_prepare, by
// rank and so in a fixed order); T and G are products over 32-token tiles of one adapter
// (k_ad_down_tiles); the wide products run on tiles of sorted tokens, gathered by
// the DMA, whose epilogue adds the adapters' term 32 tokens at a time (k_ad_matmul;
// k_ad_join where few tiles had their contraction split); dA and dB are products
// over an adapter's run of tokens (k_ad_grads).  An adapter's numbers meet only its
// own tokens: a product with another's is dropped, not multiplied by zero, so a NaN in
// one adapter stays there.
//
// Bound by the wide products: 8192 x 4096 x 11008 with 8 adapters of rank 64 takes
// 660 to 690 us (the product 600 to 690), a step of 8192 x 4096 x 4096 with 32 of rank 16
// takes 550 to 580.
#include <algorithm>

#include "common.h"
#include "gemm16.h"
#include "launch.h"

namespace qlora {

__constant__ uint32_t cAdLevel[3 * 16] = {QLORA_Q4_LEVEL_BITS};
__constant__ uint32_t cAdT8[256] = {QLORA_T8_LEVEL_BITS};

namespace {

__device__ __forceinline__ int adapter_of(const int64_t *index, int m, int n) {
  const int64_t a = index[m];
  return a >= 0 && a < n ? static_cast<int>(a) : -1;
}

}  // namespace

// ---------------------------------------------------------------------------
// Tokens sorted by adapter, in order of their number within one; tokens without
// an adapter come last.  One workgroup; wave w has the w-th part of the tokens.
//   perm [M]     token at a sorted place
//   who  [M]     its adapter, -1: none
//   seg  [n + 1] first place of every adapter's run
//   tile [ntiles] (adapter, first place, tokens <= 32, 0), ntile [1]
//   zero [64]    a row of zeros for the DMA of places past a run
namespace {
constexpr int kSortWaves = 16;
constexpr int kSortThreads = kSortWaves * 64;
constexpr int kSortBatch = 8;      // indices of a lane in flight

struct SortLds {
  int hist[kSortWaves][kAdMax + 1];
  int wsum[2][kSortWaves];
};

__device__ __forceinline__ void ad_sort(SortLds &lds, const int64_t *__restrict__ index, int M, int n, const AdPlan &p) {
  auto &hist = lds.hist;
  auto &wsum = lds.wsum;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = lane; i <= n; i += 64) hist[wave][i] = 0;
  const int per = ((M + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int lo = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(wave) * per, M));
  const int hi = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(wave + 1) * per, M));
  // Adapters of tokens m0 + lane + 64 u; -2: past this wave's part.
  auto load = [&](int (&a)[kSortBatch], int m0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      const int m = m0 + 64 * u + lane;
      const int x = adapter_of(index, min(m, M - 1), n);
      a[u] = m < hi ? x : -2;
    }
  };
  __syncthreads();
  for (int m0 = lo; m0 < hi; m0 += 64 * kSortBatch) {
    int a[kSortBatch];
    load(a, m0);
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      // the first adapter's tokens at once (runs of a prompt), the others' one by one; counts: order does not matter
      const uint64_t some = __ballot(a[u] != -2);
      if (!some) break;
      const int a0 = __builtin_amdgcn_readlane(a[u], __builtin_ctzll(some));
      const uint64_t mask = __ballot(a[u] == a0);
      if (a[u] != -2 && (a[u] != a0 || (mask & ((uint64_t{1} << lane) - 1)) == 0))
        atomicAdd(&hist[wave][a[u] < 0 ? n : a[u]], a[u] == a0 ? static_cast<int>(__popcll(mask)) : 1);
    }
  }
  if (tid < 64) p.zero[tid] = 0;
  __syncthreads();
  // Column a of the table: this adapter's tokens before each wave's part.
  int total = 0, tiles = 0;
  if (tid <= n) {
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = hist[w][tid];
      hist[w][tid] = total;
      total += c;
    }
    if (tid < n) tiles = (total + 31) / 32;
  }
  int pos = total, tpos = tiles;                 // inclusive sums over the workgroup
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(pos, o, 64), v = __shfl_up(tpos, o, 64);
    if (lane >= o) {
      pos += u;
      tpos += v;
    }
  }
  if (lane == 63) {
    wsum[0][wave] = pos;
    wsum[1][wave] = tpos;
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    pos += wsum[0][w];
    tpos += wsum[1][w];
  }
  const int start = pos - total;
  if (tid <= n) {
    for (int w = 0; w < kSortWaves; ++w) hist[w][tid] += start;
    p.seg[tid] = start;
    if (tid < n) {
      const int t0 = tpos - tiles;
      for (int i = 0; i < tiles; ++i) p.tile[t0 + i] = make_int4(tid, start + 32 * i, min(32, total - 32 * i), 0);
      if (tid == n - 1) p.ntile[0] = tpos;
    }
  }
  __syncthreads();
  for (int m0 = lo; m0 < hi; m0 += 64 * kSortBatch) {   // wave-uniform; this wave's row of the table only
    int a[kSortBatch];
    load(a, m0);
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      uint64_t left = __ballot(a[u] != -2);
      while (left) {
        const int a0 = __builtin_amdgcn_readlane(a[u], __builtin_ctzll(left));
        const uint64_t mask = __ballot(a[u] == a0);
        left &= ~mask;
        const int col = a0 < 0 ? n : a0;
        int base = 0;
        if (lane == 0) base = atomicAdd(&hist[wave][col], static_cast<int>(__popcll(mask)));
        base = __builtin_amdgcn_readfirstlane(base);
        if (a[u] == a0) {
          const int at = base + static_cast<int>(__popcll(mask & ((uint64_t{1} << lane) - 1)));
          p.perm[at] = m0 + 64 * u + lane;
          p.who[at] = a0;
        }
      }
    }
  }
}

// One R x C tile (powers of two, R C = 4096) of a matrix [rows, cols] into [cols, pitch],
// zeros in the columns rows .. pitch - 1.
constexpr int kTrTile = 256 * 17;      // R (C + 1) at most
__device__ __forceinline__ void ad_transpose(uint16_t *t, const uint16_t *__restrict__ src, int rows, int cols, int pitch, int R, int C,
                                             int r0, int c0, uint16_t *__restrict__ dst) {
  for (int i = threadIdx.x; i < 4096; i += kSortThreads) {
    const int y = i / C, x = i & (C - 1);
    t[y * (C + 1) + x] = r0 + y < rows && c0 + x < cols ? src[static_cast<int64_t>(r0 + y) * cols + c0 + x] : 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 4096; i += kSortThreads) {
    const int y = i / R, x = i & (R - 1);
    if (c0 + y < cols && r0 + x < pitch) dst[static_cast<int64_t>(c0 + y) * pitch + r0 + x] = t[x * (C + 1) + y];
  }
}

// A tile's extent along r and along the other axis: no wider than r needs (32 adapters of rank
// 16, 4096 x 4096, a step: 590 to 599 us with 64 x 64 tiles, three quarters empty, 579 so).
struct TrCut {
  int narrow, wide;
  __host__ __device__ explicit TrCut(int r) : narrow(r <= 16 ? 16 : r <= 32 ? 32 : 64), wide(4096 / narrow) {}
};
}  // namespace

// Everything that the products need beforehand and that needs nothing itself, in
// one launch: workgroup 0 sorts; the others, in this order,
//   dequantize W to bf16, as the codec does (16 codes a thread),
//   transpose A [n, r, K] -> At [n, K, r] and B [n, N, r] -> Bt [n, r, N filled up
//   to 64] (the backward products then read their adapter operand along its rows),
//   fill up dY's rows to a multiple of 64 with zeros.
// One after the other the sort, 15 us at 8192 tokens on one compute unit, and four
// launches would add up.  27 to 32 us with the 90 MB written for a weight of 4096 x 11008,
// 14 to 17 with that of 4096 x 4096 (the sort then); 8 to 13 at 777 tokens, the sort's latency.
__global__ __launch_bounds__(kSortThreads) void k_ad_prepare(const AdPrepare a) {
  __shared__ union {
    SortLds sort;
    uint16_t tile[kTrTile];
    float table[272];
  } lds;
  int b = blockIdx.x;
  if (b == 0) {
    ad_sort(lds.sort, a.index, a.M, a.n, a.plan);
    return;
  }
  b -= 1;
  if (b < a.deq) {
    float *level = lds.table, *t8 = lds.table + 16;
    if (threadIdx.x < 16) level[threadIdx.x] = u2f(cAdLevel[16 * a.w.qtype + threadIdx.x]);
    if (threadIdx.x < 256) t8[threadIdx.x] = u2f(cAdT8[threadIdx.x]);
    __syncthreads();
    const float mean = a.w.mean[0];
    const int64_t chunks = static_cast<int64_t>(a.w.N) * a.w.K / 16;   // K % 64 == 0
    for (int64_t i = static_cast<int64_t>(b) * kSortThreads + threadIdx.x; i < chunks; i += static_cast<int64_t>(a.deq) * kSortThreads) {
      const uint2 pk = *reinterpret_cast<const uint2 *>(a.w.packed + 8 * i);
      const int64_t blk = i >> 2;
      const float chat = decode_absmax(t8[a.w.code8[blk]], a.w.c2[blk >> 8], mean);
      const uint32_t words[2] = {pk.x, pk.y};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[q] = pack_bf16x2(level[(words[h] >> (8 * q)) & 15] * chat, level[(words[h] >> (8 * q + 4)) & 15] * chat);
        *reinterpret_cast<uint4 *>(a.Wd + 16 * i + 8 * h) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    return;
  }
  b -= a.deq;
  const TrCut cut(a.r);
  const int ta = (a.r + cut.narrow - 1) / cut.narrow;
  if (b < a.trA) {
    const int tk = (a.w.K + cut.wide - 1) / cut.wide;
    const int m = b / (ta * tk), j = b % (ta * tk);
    ad_transpose(lds.tile, a.A + static_cast<int64_t>(m) * a.r * a.w.K, a.r, a.w.K, a.r, cut.narrow, cut.wide, j / tk * cut.narrow,
                 j % tk * cut.wide, a.At + static_cast<int64_t>(m) * a.r * a.w.K);
    return;
  }
  b -= a.trA;
  if (b < a.trB) {
    const int tn = (a.Np + cut.wide - 1) / cut.wide;
    const int m = b / (ta * tn), j = b % (ta * tn);
    ad_transpose(lds.tile, a.B + static_cast<int64_t>(m) * a.w.N * a.r, a.w.N, a.r, a.Np, cut.wide, cut.narrow, j / ta * cut.wide,
                 j % ta * cut.narrow, a.Bt + static_cast<int64_t>(m) * a.r * a.Np);
    return;
  }
  b -= a.trB;
  const int per = a.Np >> 3;
  for (int64_t i = static_cast<int64_t>(b) * kSortThreads + threadIdx.x; i < static_cast<int64_t>(a.M) * per;
       i += static_cast<int64_t>(a.pad) * kSortThreads) {
    const int64_t m = i / per;
    const int c = 8 * static_cast<int>(i % per);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < a.w.N) v = *reinterpret_cast<const uint4 *>(a.dY + m * a.w.N + c);   // N % 8 == 0
    *reinterpret_cast<uint4 *>(a.dYp + m * a.Np + c) = v;
  }
}

// ---------------------------------------------------------------------------
// part [split][M][r] = P_m Q_a^T over 32-token tiles of one adapter and a part of the
// contraction: P [M, D] (X or dY), Q [n, r, D] (A, or B transposed).  Workgroup
// (tile, 64 adapter rows, split), 4 waves; wave w takes the 64-column steps w, w + 4, ...
// of the part from a private ring in LDS, so there is no barrier in the loop, and
// the waves are summed in wave order.  Bound by the gather of P in pieces of 128
// bytes; split so that the tiles, whose number is not a multiple of the compute units, end
// evenly.  8192 tokens, D = 11008, r = 64: 90 us unsplit, 70 to 77 in 8 parts (180 MB of P
// at 2.4 TB/s); one or two waves a workgroup, and parts for 256 to 2048 workgroups,
// are within 3 % of it in the whole layer.  r = 16, D = 4096: 20 to 24 us.
namespace {
constexpr int kDtWaves = 4;
constexpr int kDtThreads = kDtWaves * 64;
constexpr int kDtSlots = 3;

template <int kQ>
constexpr int dt_slot() { return (4 + kQ) * 1024; }   // 32 rows of P, 8 kQ rows of Q, 128 bytes each
}  // namespace

// kQ: adapter rows / 8 that are fetched (1 to 4: all of them; 8: 64 at a time, those past r repeated).
template <int kQ>
__global__ __launch_bounds__(kDtThreads) void k_ad_down_tiles(const uint16_t *__restrict__ P, int D, const uint16_t *__restrict__ Q,
                                                              int r, int M, int splits, AdPlan p, float *__restrict__ part) {
  constexpr int kJB = kQ > 4 ? 2 : 1;
  // the waves' sums at the end take 4 kJB KB; the operands of rows past 8 kQ are read from what follows a slot and not stored
  constexpr int kPad = 4096 * (1 + kJB) - dt_slot<kQ>();
  constexpr int kWaveLds = kDtSlots * dt_slot<kQ>() + kPad;
  static_assert(kWaveLds >= 4096 * kJB, "a wave's sums");
  __shared__ __attribute__((aligned(16))) uint8_t smem[kDtWaves][kWaveLds];
  if (static_cast<int>(blockIdx.x) >= p.ntile[0]) return;
  const int4 tl = p.tile[blockIdx.x];
  const int a = tl.x, p0 = tl.y, cnt = tl.z;
  const int j0 = blockIdx.y * 32 * kJB;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 31, lh = lane >> 5;
  const uint16_t *Qa = Q + static_cast<int64_t>(a) * r * D;
  const int split = blockIdx.z;
  const int first = (D >> 6) * split / splits, steps = (D >> 6) * (split + 1) / splits - first;
  const int n_i = wave < steps ? (steps - wave + kDtWaves - 1) / kDtWaves : 0;

  // 8 rows of 128 bytes a DMA instruction; the chunk that belongs at a lane's position.
  uint32_t po[4], qo[kQ];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int row = 8 * u + (lane >> 3);
    const int chunk = (lane & 7) ^ ((row & 7) ^ ((row >> 3) & 1));
    po[u] = static_cast<uint32_t>(p.perm[p0 + min(row, cnt - 1)]) * D * 2 + 16 * chunk;
  }
#pragma unroll
  for (int u = 0; u < kQ; ++u) {
    const int row = 8 * u + (lane >> 3);
    const int chunk = (lane & 7) ^ ((row & 7) ^ ((row >> 3) & 1));
    qo[u] = static_cast<uint32_t>(min(j0 + row, r - 1)) * D * 2 + 16 * chunk;   // rows past r: columns never stored
  }
  const uint32_t ring = lds_addr(smem[wave]);
  auto issue = [&](int i, int slot) __attribute__((always_inline)) {
    const int64_t k = 64 * (first + wave + static_cast<int64_t>(kDtWaves) * i);
    const uint32_t dst = __builtin_amdgcn_readfirstlane(ring + slot * dt_slot<kQ>());
#pragma unroll
    for (int u = 0; u < 4; ++u) dma16(P + k, po[u], dst + u * 1024);
#pragma unroll
    for (int u = 0; u < kQ; ++u) dma16(Qa + k, qo[u], dst + 4096 + u * 1024);
  };
  constexpr int kDma = 4 + kQ;
  f32x16_t acc[kJB];
#pragma unroll
  for (int jb = 0; jb < kJB; ++jb)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[jb][e] = 0.f;
  // Only DMAs count here: in issue order, so the two younger steps may be in flight.
  __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  if (n_i > 0) issue(0, 0);
  if (n_i > 1) issue(1, 1);
  for (int i = 0; i < n_i; ++i) {
    const int slot = i % kDtSlots;
    if (i + 2 < n_i) issue(i + 2, (i + 2) % kDtSlots);
    __builtin_amdgcn_sched_barrier(0);
    if (i + 2 < n_i)
      __builtin_amdgcn_s_waitcnt(wait_imm(2 * kDma, 15));
    else if (i + 1 < n_i)
      __builtin_amdgcn_s_waitcnt(wait_imm(kDma, 15));
    else
      __builtin_amdgcn_s_waitcnt(wait_imm(0, 15));
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t *ps = smem[wave] + slot * dt_slot<kQ>(), *qs = ps + 4096;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const bf16x8_t x = *reinterpret_cast<const bf16x8_t *>(ps + swz128(lr, 2 * s + lh));
#pragma unroll
      for (int jb = 0; jb < kJB; ++jb) {
        const bf16x8_t y = *reinterpret_cast<const bf16x8_t *>(qs + swz128(32 * jb + lr, 2 * s + lh));
        acc[jb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, acc[jb], 0, 0, 0);
      }
    }
    // The operand reads are done before the next step's DMA into this slot is issued.
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_imm(63, 0));
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
  }
  // lane: column (adapter row) lr of block jb, token 8 (e / 4) + 4 lh + e % 4.
  float *red = reinterpret_cast<float *>(smem[wave]);
#pragma unroll
  for (int jb = 0; jb < kJB; ++jb)
#pragma unroll
    for (int e = 0; e < 16; ++e) red[(8 * (e >> 2) + 4 * lh + (e & 3)) * 32 * kJB + 32 * jb + lr] = acc[jb][e];
  __syncthreads();
  for (int idx = threadIdx.x; idx < 32 * 8 * kJB; idx += kDtThreads) {
    const int row = idx / (8 * kJB), c = idx % (8 * kJB), j = j0 + 4 * c;
    if (row >= cnt || j >= r) continue;          // r % 8 == 0
    f32x4_t v = reinterpret_cast<const f32x4_t *>(smem[0])[row * 8 * kJB + c];
#pragma unroll
    for (int w = 1; w < kDtWaves; ++w) v += reinterpret_cast<const f32x4_t *>(smem[w])[row * 8 * kJB + c];
    *reinterpret_cast<f32x4_t *>(part + (static_cast<int64_t>(split) * M + p.perm[p0 + row]) * r + j) = v;
  }
}

// out [M, r] = bf16(scale_a times the sum of the parts), 0 for tokens without an
// adapter; all parts' loads at once (3 to 6 us: its launch, and 17 MB at r = 64).
__global__ __launch_bounds__(256) void k_ad_sum(const float *__restrict__ part, int splits, int M, int r, const int64_t *__restrict__ index,
                                                int n, const float *__restrict__ scale, uint16_t *__restrict__ out) {
  const int64_t all = static_cast<int64_t>(M) * r;
  const int64_t i = 4 * (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x);
  if (i >= all) return;
  const int a = adapter_of(index, static_cast<int>(i / r), n);
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (a >= 0) {
    f32x4_t q[kAdSplits];
#pragma unroll
    for (int s = 0; s < kAdSplits; ++s) q[s] = *reinterpret_cast<const f32x4_t *>(part + min(s, splits - 1) * all + i);
#pragma unroll
    for (int s = 0; s < kAdSplits; ++s)
      if (s < splits) v += q[s];
    const float sc = scale[a];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= sc;
  }
  *reinterpret_cast<uint2 *>(out + i) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// ---------------------------------------------------------------------------
// C [M, cols] = L Wd^T (or L Wd) + T_m U_a^T: L = X, U = B (NT), or L = dY, U
// = A transposed (NN); U [n, cols, r].  The adapters' term is added to a
// wave's accumulators 32 tokens at a time, from T and U as they lie in memory (16
// bytes a lane are an operand of the matrix instruction).  Sorted tokens: most
// blocks have one adapter and accumulate in place; in the others the product is
// formed apart and added in the lanes whose token has this adapter.
// 8192 tokens: 600 to 690 us for 4096 x 11008 (1.07 to 1.23 PFLOP/s), 231 to 246 for 4096 x
// 4096, 236 to 268 for its NN form.
// Kc, L's row pitch: a multiple of 64; NN: columns N .. Kc - 1 of L are zero.
namespace {
struct AdMatmul {
  const uint16_t *L, *Wd, *T, *U;
  uint16_t *out;
  float *part;       // [split][tile][...] where the contraction is split
  AdPlan p;
  int Kc, M, N, K, r, cols, splits;
};

// Adds the adapters' term to a tile's accumulators and stores them.
template <class S>
__device__ __forceinline__ void ad_finish(const AdMatmul &g, int m0, int c0, uint8_t *smem, gemm16::Acc<S> &acc) {
  using namespace gemm16;
  const int M = g.M, cols = g.cols, r = g.r;
  const AdPlan &p = g.p;
  const Place<S> w;
  const int lr = w.lr, lh = w.lh, cw = c0 + w.col0();
  static_assert(S::kFN == 2, "two column fragments a wave");
#pragma unroll
  for (int i = 0; i < S::kFM; ++i) {
    const int at = min(m0 + w.row0() + 32 * i + lr, M - 1);
    const int a = p.who[at];
    const uint16_t *trow = g.T + static_cast<int64_t>(p.perm[at]) * r;
    uint64_t left = __ballot(a >= 0);
    while (left) {
      const int a0 = __builtin_amdgcn_readlane(a, __builtin_ctzll(left));
      const uint64_t mask = __ballot(a == a0);
      left &= ~mask;
      const uint16_t *u0 = g.U + (static_cast<int64_t>(a0) * cols + min(cw + lr, cols - 1)) * r;
      const uint16_t *u1 = g.U + (static_cast<int64_t>(a0) * cols + min(cw + 32 + lr, cols - 1)) * r;
      const bool whole = mask == ~uint64_t{0};
      f32x16_t part[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) part[j][e] = whole ? acc[i][j][e] : 0.f;
      for (int j0 = 0; j0 < r; j0 += 16) {
        const int j = j0 + 8 * lh;
        const bool ok = j < r;                    // r % 8 == 0
        bf16x8_t tv = *reinterpret_cast<const bf16x8_t *>(trow + (ok ? j : 0));
        bf16x8_t v0 = *reinterpret_cast<const bf16x8_t *>(u0 + (ok ? j : 0));
        bf16x8_t v1 = *reinterpret_cast<const bf16x8_t *>(u1 + (ok ? j : 0));
        if (!ok) tv = v0 = v1 = bf16x8_t{};
        part[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v0, tv, part[0], 0, 0, 0);
        part[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v1, tv, part[1], 0, 0, 0);
      }
      const bool mine = a == a0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = whole ? part[j][e] : acc[i][j][e] + (mine ? part[j][e] : 0.f);
    }
  }
  store_bf16<S>(acc, smem, [&](int row, int col, uint4 v) {
    if (m0 + row < M && c0 + col < cols)          // cols % 8 == 0
      *reinterpret_cast<uint4 *>(g.out + static_cast<int64_t>(p.perm[m0 + row]) * cols + c0 + col) = v;
  });
}

// A wave's accumulators of a split of a tile, as its lanes hold them.
template <class S>
__device__ __forceinline__ f32x4_t *ad_part(const AdMatmul &g, int split, int tile, int tiles) {
  return reinterpret_cast<f32x4_t *>(g.part + (static_cast<int64_t>(split) * tiles + tile) * S::kBM * S::kBN) +
         static_cast<int64_t>(threadIdx.x >> 6) * (S::kWaveRows * S::kWaveCols / 4) + (threadIdx.x & 63);
}
}  // namespace

template <class S, bool kNN, bool kSplit>
__global__ __launch_bounds__(S::kThreads, 2) void k_ad_matmul(const AdMatmul g) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[S::kLds];
  const int trows = (g.M + S::kBM - 1) / S::kBM, tcols = (g.cols + S::kBN - 1) / S::kBN, tiles = trows * tcols;
  const int split = kSplit ? blockIdx.x / tiles : 0, id = blockIdx.x - split * tiles;
  int tr, tc;
  if (!place(id, trows, tcols, tr, tc)) return;
  const int m0 = tr * S::kBM, c0 = tc * S::kBN;
  const int KT = g.Kc / kBK;
  const int k0 = kSplit ? KT * split / g.splits : 0, k1 = kSplit ? KT * (split + 1) / g.splits : KT;   // KT >= 8 splits
  Acc<S> acc;
  tile<S, kNN>(smem, g.L + kBK * k0, g.Kc, [&](int row) { return g.p.perm[min(m0 + row, g.M - 1)]; },
               kNN ? g.Wd + static_cast<int64_t>(kBK) * k0 * g.K : g.Wd + kBK * k0, g.K, c0, g.cols - 1, g.N - 1 - kBK * k0, k1 - k0, acc);
  if constexpr (!kSplit) {
    ad_finish<S>(g, m0, c0, smem, acc);
  } else {
    f32x4_t *part = ad_part<S>(g, split, tr * tcols + tc, tiles);
#pragma unroll
    for (int i = 0; i < S::kFM; ++i)
#pragma unroll
      for (int j = 0; j < S::kFN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          part[64 * (4 * (S::kFN * i + j) + q)] = f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  }
}

// A tile's splits added in order, then as above (105 x 3232 x 10944: the layer takes 56 us
// with the contraction split and this launch, 179 without).
template <class S>
__global__ __launch_bounds__(S::kThreads, 2) void k_ad_join(const AdMatmul g) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[S::kLds];
  const int tcols = (g.cols + S::kBN - 1) / S::kBN;
  const int tr = blockIdx.x / tcols, tc = blockIdx.x % tcols;
  Acc<S> acc;
  clear<S>(acc);
  for (int s = 0; s < g.splits; ++s) {
    const f32x4_t *part = ad_part<S>(g, s, blockIdx.x, gridDim.x);
#pragma unroll
    for (int i = 0; i < S::kFM; ++i)
#pragma unroll
      for (int j = 0; j < S::kFN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t v = part[64 * (4 * (S::kFN * i + j) + q)];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
        }
  }
  ad_finish<S>(g, tr * S::kBM, tc * S::kBN, smem, acc);
}

// ---------------------------------------------------------------------------
// dA_a [r, K] = sum G_m^T X_m and dB_a [N, r] = sum dY_m^T T_m over an adapter's
// run: acc[j][d] = sum_m Q[m][j] P[m][d] for 64 columns d of the wide operand
// and 32 kJB columns j of the narrow one.  Workgroup (64-column chunk of X or
// dY, adapter, chunk of r); wave w takes 32-token stages w, w + 4, ... of the run
// in a private ring; both operands are read with the transposing LDS load.
// Places past the run are read from a row of zeros.  Empty runs give zeros.  Short
// runs take 2 waves: a workgroup then has 37 KB of LDS and a compute unit four of them,
// over whose starts and ends the others work.  Bound by reading X and dY, 134 MB at
// 8192 x (4096 + 4096): 29 us where the caches hold part of it, 45 in a step (3 TB/s).
// Those are even runs of 32 adapters.  A run is not divided, and the waves go by the average
// run: 101 us where one of the 32 has all 8192 tokens (two waves; 46 to 51 where it is the
// only one held, four waves), and at 1024 + 1024 columns, 64 adapters, 78 against 13.
namespace {
constexpr int kGdTile = 32 * 128;
constexpr int kGdSlot = 2 * kGdTile;   // P then Q
constexpr int kGdChunk = 1024;         // places whose tokens are held in LDS at a time

// Byte offset in a [32 tokens][64 columns] swizzled tile of this lane's
// source for the transposed read that hands lanes 16 G .. +15 columns
// 32 cb + 16 (G % 2) .. +15 of tokens 8 (G / 2) + 4 h .. +3 (+ 16 s).
__device__ __forceinline__ uint32_t gd_offset(int lane, int cb, int h) {
  const int t = lane & 15, g = lane >> 4;
  const int row = 8 * (g >> 1) + 4 * h + (t >> 2);
  const int chunk = 4 * cb + 2 * (g & 1) + ((t & 3) >> 1);
  return static_cast<uint32_t>(swz128(row, chunk) + 8 * (t & 1));
}
}  // namespace

struct AdGradArgs {
  const uint16_t *P[2], *Q[2];
  uint16_t *out[2];
  int D[2], chunks[2];   // columns of P; 64-column chunks (0: not wanted)
  int r;
};

template <int kGdWaves>
__global__ __launch_bounds__(kGdWaves * 64) void k_ad_grads(AdGradArgs g, AdPlan p) {
  constexpr int kGdThreads = kGdWaves * 64;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kGdWaves][2][kGdSlot];
  __shared__ int sTok[kGdChunk];
  const int which = static_cast<int>(blockIdx.x) < g.chunks[0] ? 0 : 1;
  const int d0 = 64 * (static_cast<int>(blockIdx.x) - (which ? g.chunks[0] : 0));
  const int a = blockIdx.y, j0 = 64 * blockIdx.z;
  const uint16_t *P = g.P[which], *Q = g.Q[which];
  const int D = g.D[which], r = g.r;
  const int s0 = p.seg[a], s1 = p.seg[a + 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 31, lh = lane >> 5;
  const uint32_t ring = lds_addr(smem[wave][0]);
  const bool two = r - j0 > 32;
  f32x16_t acc[2][2];   // [j block][d block]
#pragma unroll
  for (int jb = 0; jb < 2; ++jb)
#pragma unroll
    for (int db = 0; db < 2; ++db)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[jb][db][e] = 0.f;
  uint32_t off[2][2];
#pragma unroll
  for (int cb = 0; cb < 2; ++cb)
#pragma unroll
    for (int h = 0; h < 2; ++h) off[cb][h] = gd_offset(lane, cb, h);
  auto operand = [&](const uint8_t *t, int cb, int s) __attribute__((always_inline)) {
    const gemm16::bf16x4_t lo = gemm16::ds_tr16(t + off[cb][0] + 2048 * s);
    const gemm16::bf16x4_t hi = gemm16::ds_tr16(t + off[cb][1] + 2048 * s);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  for (int c0 = s0; c0 < s1; c0 += kGdChunk) {
    const int places = min(kGdChunk, s1 - c0), stages = (places + 31) >> 5;
    for (int i = threadIdx.x; i < 32 * stages; i += kGdThreads) sTok[i] = i < places ? p.perm[c0 + i] : -1;
    __syncthreads();
    const int n_i = wave < stages ? (stages - wave + kGdWaves - 1) / kGdWaves : 0;
    auto issue = [&](int i, int slot) __attribute__((always_inline)) {
      const uint32_t dst = __builtin_amdgcn_readfirstlane(ring + slot * kGdSlot);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = 8 * u + (lane >> 3);
        const int chunk = (lane & 7) ^ ((row & 7) ^ ((row >> 3) & 1));
        const int m = sTok[32 * (wave + kGdWaves * i) + row];
        const int dc = min(d0 + 8 * chunk, D - 8);    // D % 8 == 0: columns past it are never stored
        const int jc = min(j0 + 8 * chunk, r - 8);
        const uint16_t *ps = m >= 0 ? P + static_cast<int64_t>(m) * D + dc : p.zero;
        const uint16_t *qs = m >= 0 ? Q + static_cast<int64_t>(m) * r + jc : p.zero;
        dma16(ps, dst + u * 1024);
        dma16(qs, dst + kGdTile + u * 1024);
      }
    };
    if (n_i > 0) issue(0, 0);
    for (int i = 0; i < n_i; ++i) {
      const int slot = i & 1;
      if (i + 1 < n_i) issue(i + 1, slot ^ 1);
      __builtin_amdgcn_sched_barrier(0);
      if (i + 1 < n_i)
        __builtin_amdgcn_s_waitcnt(wait_imm(8, 15));
      else
        __builtin_amdgcn_s_waitcnt(wait_imm(0, 15));
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_sched_barrier(0);
      const uint8_t *ps = smem[wave][slot], *qs = ps + kGdTile;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bf16x8_t x0 = operand(ps, 0, s), x1 = operand(ps, 1, s);
        const bf16x8_t q0 = operand(qs, 0, s);
        acc[0][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q0, x0, acc[0][0], 0, 0, 0);
        acc[0][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q0, x1, acc[0][1], 0, 0, 0);
        if (two) {
          const bf16x8_t q1 = operand(qs, 1, s);
          acc[1][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q1, x0, acc[1][0], 0, 0, 0);
          acc[1][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q1, x1, acc[1][1], 0, 0, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_imm(63, 0));   // operand reads done before the slot is filled again
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();                                  // sTok has been read
  }
  // lane: column d = lr of block db, row j = 8 (e / 4) + 4 lh + e % 4 of block jb.
  // Sums over the waves in LDS, one j block (32 x 64 fp32) at a time.
  for (int jb = 0; jb < (two ? 2 : 1); ++jb) {
    float *red = reinterpret_cast<float *>(smem[wave][0]);
#pragma unroll
    for (int db = 0; db < 2; ++db)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        red[(8 * (e >> 2) + 4 * lh + (e & 3)) * 64 + 32 * db + lr] = jb ? acc[1][db][e] : acc[0][db][e];
    __syncthreads();
    auto sum = [&](int j, int d) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kGdWaves; ++w) v += reinterpret_cast<const float *>(smem[w][0])[j * 64 + d];
      return v;
    };
    const int jr = min(32, r - j0 - 32 * jb);     // rows of this block, a multiple of 8
    if (which == 0) {                             // [r][D]
      for (int idx = threadIdx.x; idx < jr * 8; idx += kGdThreads) {
        const int j = idx >> 3, d = 8 * (idx & 7);
        if (d0 + d >= D) continue;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = sum(j, d + q);
        *reinterpret_cast<uint4 *>(g.out[0] + (static_cast<int64_t>(a) * r + j0 + 32 * jb + j) * D + d0 + d) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      }
    } else {                                      // [D][r]
      for (int idx = threadIdx.x; idx < 64 * (jr >> 3); idx += kGdThreads) {
        const int d = idx / (jr >> 3), j = 8 * (idx % (jr >> 3));
        if (d0 + d >= D) continue;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = sum(j + q, d);
        *reinterpret_cast<uint4 *>(g.out[1] + (static_cast<int64_t>(a) * D + d0 + d) * r + j0 + 32 * jb + j) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
hipError_t launch_ad_prepare(AdPrepare a, hipStream_t s) {
  const TrCut cut(a.r);
  const int ta = (a.r + cut.narrow - 1) / cut.narrow, tk = (a.w.K + cut.wide - 1) / cut.wide, tn = (a.Np + cut.wide - 1) / cut.wide;
  const int64_t chunks = static_cast<int64_t>(a.w.N) * a.w.K / 16;
  a.deq = a.Wd ? static_cast<int>(std::min<int64_t>(2048, (chunks + kSortThreads - 1) / kSortThreads)) : 0;
  a.trA = a.At ? a.n * ta * tk : 0;
  a.trB = a.Bt ? a.n * ta * tn : 0;
  a.pad = a.dYp ? static_cast<int>(std::min<int64_t>(1024, (static_cast<int64_t>(a.M) * a.Np / 8 + kSortThreads - 1) / kSortThreads)) : 0;
  hipLaunchKernelGGL(k_ad_prepare, dim3(1 + a.deq + a.trA + a.trB + a.pad), dim3(kSortThreads), 0, s, a);
  return hipGetLastError();
}

int ad_down_splits(int64_t M, int64_t D, int n) {
  const int64_t tiles = ad_tiles_max(M, n);
  // about four workgroups a compute unit, at least 8 steps each
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kAdSplits, (1024 + tiles - 1) / tiles, D / 64 / 8})));
}

hipError_t launch_ad_down(const uint16_t *P, int M, int D, const uint16_t *Q, const AdapterSet &ad, const AdPlan &p, float *part,
                          uint16_t *out, hipStream_t s) {
  const int tiles = static_cast<int>(ad_tiles_max(M, ad.n)), splits = ad_down_splits(M, D, ad.n);
  const dim3 grid(tiles, (ad.r + 63) / 64, splits), th(kDtThreads);
  switch (ad.r <= 32 ? ad.r / 8 : 8) {
    case 1: hipLaunchKernelGGL(k_ad_down_tiles<1>, grid, th, 0, s, P, D, Q, ad.r, M, splits, p, part); break;
    case 2: hipLaunchKernelGGL(k_ad_down_tiles<2>, grid, th, 0, s, P, D, Q, ad.r, M, splits, p, part); break;
    case 3: hipLaunchKernelGGL(k_ad_down_tiles<3>, grid, th, 0, s, P, D, Q, ad.r, M, splits, p, part); break;
    case 4: hipLaunchKernelGGL(k_ad_down_tiles<4>, grid, th, 0, s, P, D, Q, ad.r, M, splits, p, part); break;
    default: hipLaunchKernelGGL(k_ad_down_tiles<8>, grid, th, 0, s, P, D, Q, ad.r, M, splits, p, part); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t quads = static_cast<int64_t>(M) * ad.r / 4;
  hipLaunchKernelGGL(k_ad_sum, dim3(static_cast<unsigned>((quads + 255) / 256)), dim3(256), 0, s, part, splits, M, ad.r, ad.index, ad.n,
                     ad.scale, out);
  return hipGetLastError();
}

namespace {
using gemm16::Big;
using gemm16::Deep;
using gemm16::Mid;
template <class S>
int tiles_of(int64_t M, int64_t cols) {
  return static_cast<int>((M + S::kBM - 1) / S::kBM * ((cols + S::kBN - 1) / S::kBN));
}
}  // namespace

// Splits of the contraction for products of few tiles: as many as give every
// compute unit a workgroup, 8 steps each at least.
int ad_matmul_splits(int64_t M, int64_t cols, int64_t Kc) {
  if (!gemm16::use_mid(M, cols) || !gemm16::use_deep(M, cols)) return 1;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({256 / tiles_of<Deep>(M, cols), Kc / 64 / 8, 16})));
}
size_t ad_matmul_part_floats(int64_t M, int64_t cols, int64_t Kc) {
  const int splits = ad_matmul_splits(M, cols, Kc);
  return splits > 1 ? static_cast<size_t>(splits) * tiles_of<Deep>(M, cols) * Deep::kBM * Deep::kBN : 0;
}

template <bool kNN>
static hipError_t launch_ad_matmul(AdMatmul g, hipStream_t s) {
  g.cols = kNN ? g.K : g.N;
  g.splits = ad_matmul_splits(g.M, g.cols, g.Kc);
  if (!gemm16::use_mid(g.M, g.cols)) {
    hipLaunchKernelGGL((k_ad_matmul<Big, kNN, false>), dim3(tiles_of<Big>(g.M, g.cols)), dim3(Big::kThreads), 0, s, g);
    return hipGetLastError();
  }
  const int tiles = tiles_of<Deep>(g.M, g.cols);
  if (!gemm16::use_deep(g.M, g.cols)) {
    hipLaunchKernelGGL((k_ad_matmul<Mid, kNN, false>), dim3(tiles), dim3(Mid::kThreads), 0, s, g);
    return hipGetLastError();
  }
  if (g.splits == 1) {
    hipLaunchKernelGGL((k_ad_matmul<Deep, kNN, false>), dim3(tiles), dim3(Deep::kThreads), 0, s, g);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_ad_matmul<Deep, kNN, true>), dim3(tiles * g.splits), dim3(Deep::kThreads), 0, s, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_ad_join<Deep>, dim3(tiles), dim3(Deep::kThreads), 0, s, g);
  return hipGetLastError();
}
hipError_t launch_ad_matmul_fwd(const uint16_t *X, int M, int N, int K, const uint16_t *Wd, const uint16_t *T, const uint16_t *B, int r,
                                const AdPlan &p, float *part, uint16_t *Y, hipStream_t s) {
  return launch_ad_matmul<false>(AdMatmul{X, Wd, T, B, Y, part, p, K, M, N, K, r, 0, 0}, s);
}
hipError_t launch_ad_matmul_dx(const uint16_t *dY, int Np, int M, int N, int K, const uint16_t *Wd, const uint16_t *G,
                               const uint16_t *At, int r, const AdPlan &p, float *part, uint16_t *dX, hipStream_t s) {
  return launch_ad_matmul<true>(AdMatmul{dY, Wd, G, At, dX, part, p, Np, M, N, K, r, 0, 0}, s);
}

hipError_t launch_ad_grads(const uint16_t *X, const uint16_t *dY, const uint16_t *G, const uint16_t *T, int M, int N, int K, const AdapterSet &ad,
                           const AdPlan &p, uint16_t *dA, uint16_t *dB, hipStream_t s) {
  AdGradArgs g{{X, dY}, {G, T}, {dA, dB}, {K, N}, {dA ? (K + 63) / 64 : 0, dB ? (N + 63) / 64 : 0}, ad.r};
  const dim3 grid(g.chunks[0] + g.chunks[1], ad.n, (ad.r + 63) / 64);
  if (static_cast<int64_t>(M) < 1024 * static_cast<int64_t>(ad.n))
    hipLaunchKernelGGL(k_ad_grads<2>, grid, dim3(128), 0, s, g, p);
  else
    hipLaunchKernelGGL(k_ad_grads<4>, grid, dim3(256), 0, s, g, p);
  return hipGetLastError();
}

}  // namespace qlora
