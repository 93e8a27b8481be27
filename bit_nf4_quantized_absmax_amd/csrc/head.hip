// Softmax cross entropy through a frozen output head on gfx950, without the logits:
//     z = X W^T        loss_m = log sum_j e^z_mj - z_m,t      t = target[m]
//     dX = dz W        dW = dz^T X        dz_mj = weight_m (p_mj - [j = t])
//
// The vocabulary is taken in pieces.  A tile of a piece's logits
// (k_head_logits) is turned into E = e^(z - ref) and its row sums before it leaves
// the registers; E is rounded to bf16, and the sum over the piece of E W is added
// to the gradient in fp32 (k_head_acc): two products in all for loss and dX, as
// the sum over the rows of W weighted by e^z needs no division before its end.
//
//  * ref is the multiple of 64 ln 2 nearest to the largest logit of a row's 64
//    words, so that hardly ever two groups of words of a row differ in it: e^22, and
//    what lies 65 below the largest, fit into fp32 and bf16 alike, whose relative
//    precision does not depend on the scale.  Where they differ, the sums and E are
//    brought to the largest (k_head_refs; E by a power of 2^64, which rounds
//    nothing a second time), and the gradient so far by the next product's epilogue.
//  * The target's own term is left out of E and of the sums, and joins them in 64
//    bits at the end (k_head_finish): the loss is log(1 + sum / e^(z_t - ref)), and
//    (p_t - 1) W_t is added in fp32, where a rounded p_t near 1 would lose both.  E's
//    rounding to bf16 is the operand type of the second product; its error is that of
//    one output rounding, averaged over words.
//  * Rows without a target take no part: the rows that have one are listed
//    first (k_head_rows), and the DMA gathers them; for dW, where they are the
//    contraction, they are copied together (k_head_gather).
//  * dW, where the head is tuned as well, makes its logits a second time, for
//    dz needs the whole row's sum: dz^T piece by piece in bf16 (k_head_dz), then
//    dz^T X (k_head_dw).  p_t - 1 of a sure target comes from the loss there, too, which
//    the row's pair for the log-sum-exp holds (RowResult).
//  * Bound by the two (with dW four) products: 8192 x 32000 x 4096 with 6144 targets takes
//    2770 us (1.16 PFLOP/s over the whole call), 2048 x 131072 x 4096 with dW
//    7500 (1.17); few rows by reading W, 58 us for one of 32000 x 4096 (4.6 TB/s).
#include <algorithm>

#include "common.h"
#include "gemm16.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kBucket = 44.361419555836498f;   // 64 ln 2
constexpr float kWide = 0x1p20f;                 // above it a multiple of kBucket has no bits left to be near anything
constexpr float kSure = 0.5f;                    // losses below it: p_t above 0.6
constexpr float kNoLoss = 0x1p-126f;             // stands for a loss of 0 (or below it) where a positive one is needed

// e^x through the hardware's 2^x (x <= 23 here; what underflows is 0).
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// The reference of words whose largest logit is top; 0 where that is no number.
__device__ __forceinline__ float ref_of(float top) {
  if (!(fabsf(top) <= 3.0e38f)) return 0.f;
  return fabsf(top) < kWide ? kBucket * rintf(top * (1.f / kBucket)) : top;
}

// e^(from - to) for values that are rounded to bf16 already: between two multiples of kBucket (as fp32 holds them) a power of 2^64.
__device__ __forceinline__ float shift_of(float from, float to) {
  if (fabsf(from) < kWide && fabsf(to) < kWide) return __builtin_amdgcn_exp2f(64.f * rintf((from - to) * (1.f / kBucket)));
  return exp_f(from - to);
}

// Splits of the second product's words: the fewest that come within 2 % of the
// least time, in rounds of the workgroups that the chip holds at once and the
// writing and reading of a split's sums (cut.cost of a round of the whole words).
// The number of rows that count is known on the device alone.  slots 0: all of them.
__host__ __device__ __forceinline__ int splits_for(int tiles, const HeadCut &cut) {
  if (cut.slots == 0) return cut.most;
  int best = 1;
  float least = 3.4e38f;
  for (int s = 1; s <= cut.most; ++s) {
    const float t = static_cast<float>((tiles * s + cut.slots - 1) / cut.slots) / s + cut.cost * tiles * s;
    if (t < 0.98f * least) {
      least = t;
      best = s;
    }
  }
  return best;
}

// A row's loss and log-sum-exp from the sum s of all words but the target at a
// reference (0: there are none) and the target's logit; inv: 1 / the whole sum at that reference.
// The log-sum-exp is a pair that sums to it: (reference, rest), or where the target is sure
// (loss, target's logit), from which dW takes p_t - 1 = expm1(-loss) without a
// difference of two numbers near 1.  The loss is told from a reference by lying in (0, kSure): a
// reference is 0, a multiple of kBucket or beyond kWide.
struct RowResult {
  float loss, inv, lse[2];
  __device__ __forceinline__ RowResult(double s, float zt, float at) {
    const double u = static_cast<double>(at) - zt;
    double l = s == 0.0 ? 0.0 : u > 0.0 ? u + log(s + exp(-u)) : log1p(s * exp(u));
    if (!(fabsf(zt) < INFINITY) || !(s < INFINITY)) l = NAN;
    inv = s == 0.0 ? 0.f : static_cast<float>(exp(u - l));
    loss = static_cast<float>(l);
    if (loss < kSure) {
      lse[0] = fmaxf(loss, kNoLoss);
      lse[1] = zt;
    } else {
      lse[0] = static_cast<double>(zt) > static_cast<double>(at) + kBucket ? ref_of(zt) : at;
      lse[1] = static_cast<float>(l + (static_cast<double>(zt) - lse[0]));
    }
  }
};

// *at = v, or f *at + v.
__device__ __forceinline__ void add_to(f32x4_t *at, f32x4_t v, int first, float f) {
  if (!first) {
    const f32x4_t o = *at;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += f * o[e];
  }
  *at = v;
}

__device__ __forceinline__ float swap_halves(float v) { return __shfl_xor(v, 32, 64); }

}  // namespace

// ---------------------------------------------------------------------------
// Rows with a target, in order: list [count] of row numbers, tgt [count], place
// [M] of a row in the list (-1: none).  One workgroup.
__global__ __launch_bounds__(1024) void k_head_rows(const int64_t *__restrict__ target, int M, int V, HeadRows h) {
  __shared__ int wsum[2][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kBatch = 8;                          // targets of a thread in flight
  int base = 0;
  for (int64_t b0 = 0; b0 < M; b0 += 1024 * kBatch) {
    int64_t t[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t m = b0 + 1024 * u + threadIdx.x;
      t[u] = target[m < M ? m : M - 1];
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t m = b0 + 1024 * u + threadIdx.x;
      if (b0 + 1024 * u >= M) break;                 // uniform
      const bool real = m < M && t[u] >= 0 && t[u] < V;
      const uint64_t mask = __ballot(real);
      if (lane == 0) wsum[u & 1][wave] = __popcll(mask);
      __syncthreads();                               // one a round: the sums alternate
      int before = base, all = 0;
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        const int x = wsum[u & 1][w];
        if (w < wave) before += x;
        all += x;
      }
      const int at = before + static_cast<int>(__popcll(mask & ((uint64_t{1} << lane) - 1)));
      if (m < M) h.place[m] = real ? at : -1;
      if (real) {
        h.list[at] = static_cast<int>(m);
        h.tgt[at] = static_cast<int>(t[u]);
      }
      base += all;
    }
  }
  if (threadIdx.x == 0) h.count[0] = base;
}

// Xc [count filled up to 64][K]: the listed rows of X, zeros behind; twice: the same again behind them.
__global__ __launch_bounds__(256) void k_head_gather(const uint16_t *__restrict__ X, int K, HeadRows h, int twice, uint16_t *__restrict__ Xc) {
  const int count = h.count[0], rows = (count + 63) / 64 * 64, per = K >> 3;
  const int64_t all = static_cast<int64_t>(rows) * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int row = static_cast<int>(i / per), c = static_cast<int>(i % per);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < count) v = *reinterpret_cast<const uint4 *>(X + static_cast<int64_t>(h.list[row]) * K + 8 * c);
    *reinterpret_cast<uint4 *>(Xc + static_cast<int64_t>(row) * K + 8 * c) = v;
    if (twice) *reinterpret_cast<uint4 *>(Xc + static_cast<int64_t>(rows + row) * K + 8 * c) = v;
  }
}

// ---------------------------------------------------------------------------
// Words v0 .. v0 + words - 1 of the listed rows: part [64-word group][row] =
// (ref, sum of e^(z - ref)) without the target, the target's logit where it is
// among them, and with kE the matrix E [row][pitch], pitch = words filled up to 64,
// zero there and at the target.  6144 rows x 16384 words x 4096: 667 to 703 us (1.17 to 1.24
// PFLOP/s).  225 rows x 50001 x 1088, one row of tiles: 35 us (3.7 TB/s of W and E).
template <class S, bool kE>
__global__ __launch_bounds__(S::kThreads, 2) void k_head_logits(const uint16_t *__restrict__ X, const uint16_t *__restrict__ W, int K,
                                                                  int v0, int words, HeadRows h, HeadPiece pc) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[S::kLds];
  const int count = h.count[0];
  int tr, tc;
  if (!place(blockIdx.x, (count + S::kBM - 1) / S::kBM, (words + S::kBN - 1) / S::kBN, tr, tc)) return;
  const int m0 = tr * S::kBM, c0 = tc * S::kBN;
  Acc<S> acc;
  tile<S, false>(smem, X, K, [&](int row) { return h.list[min(m0 + row, count - 1)]; }, W + static_cast<int64_t>(v0) * K, K, c0,
                 words - 1, 0, K / kBK, acc);
  const Place<S> w;
  const int lr = w.lr, lh = w.lh;
  const int cw = c0 + w.col0();                       // first word (of the piece) of this wave
  const bool edge = cw + 64 > words;
#pragma unroll
  for (int i = 0; i < S::kFM; ++i) {
    const int row = m0 + w.row0() + 32 * i + lr;
    const bool live = row < count;
    const int rel = live ? h.tgt[row] - v0 - cw - 4 * lh : -1;   // of this half's words: 0 .. 3, 8 .. 11, ...
    if (edge) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (cw + 32 * j + 8 * (e >> 2) + 4 * lh + (e & 3) >= words) acc[i][j][e] = -INFINITY;
    }
    const bool hit = rel >= 0 && rel < 64 && (rel & 4) == 0;
    if (__ballot(hit) != 0) {                          // the target: kept, and out of the words
      float zt = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (rel == 32 * j + 8 * (e >> 2) + (e & 3)) {
            zt = acc[i][j][e];
            acc[i][j][e] = -INFINITY;
          }
      if (hit) h.zt[row] = zt;
    }
    float top = acc[i][0][0];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][j][e]);
    top = fmaxf(top, swap_halves(top));
    const float ref = ref_of(top);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = exp_f(acc[i][j][e] - ref);
        sum += x;
        acc[i][j][e] = x;
      }
    sum += swap_halves(sum);
    if (live && lh == 0 && cw < words) pc.part[static_cast<int64_t>(cw >> 6) * pc.rows + row] = make_float2(ref, sum);
  }
  if constexpr (kE)
    store_bf16<S>(acc, smem, [&](int row, int col, uint4 v) {
      if (m0 + row < count && c0 + col < pc.pitch)
        *reinterpret_cast<uint4 *>(pc.E + static_cast<int64_t>(m0 + row) * pc.pitch + c0 + col) = v;
    });
}

// ---------------------------------------------------------------------------
// A row's sum with this piece's groups, at the largest of their references and
// its own so far: ref and sum [row], factor [row] = e^(old ref - ref) for the
// gradient so far (0 at the first piece).  Groups of E at a smaller reference are
// brought to this one, in a second pass that hardly any row needs.  Workgroup:
// kRows rows, 256 / kRows threads share a row's groups.
template <int kRows>
__global__ __launch_bounds__(256) void k_head_refs(HeadRows h, HeadPiece pc, int groups, int first, int scale_e, float *__restrict__ loss,
                                                   float *__restrict__ lse) {
  constexpr int kShare = 256 / kRows;
  __shared__ float sRef[4][kRows], sLow[4][kRows];
  __shared__ double sSum[4][kRows];
  const int lrow = threadIdx.x % kRows, w = threadIdx.x / kRows;
  const int count = h.count[0];
  int row = blockIdx.x * kRows + lrow;
  if (loss) {                                        // kRows == 1: a workgroup a row of X
    row = h.place[blockIdx.x];
    if (row < 0) {
      if (threadIdx.x == 0) loss[blockIdx.x] = lse[2 * blockIdx.x] = lse[2 * blockIdx.x + 1] = 0.f;
      return;
    }
  } else if (static_cast<int>(blockIdx.x) * kRows >= count) {
    return;
  }
  const bool live = row < count;
  const float2 *part = pc.part + (live ? row : 0);
  const int64_t pitch = pc.rows;
  float ref = -3.4e38f, low = 3.4e38f;
  double sum = 0.0;
  constexpr int kBatch = 8;
  for (int g0 = w; g0 < groups; g0 += kShare * kBatch) {
    float2 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) v[u] = part[pitch * min(g0 + kShare * u, groups - 1)];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (g0 + kShare * u >= groups || v[u].y == 0.f) continue;
      low = fminf(low, v[u].x);
      if (v[u].x > ref) {
        sum *= exp_f(ref - v[u].x);
        ref = v[u].x;
      }
      sum += static_cast<double>(v[u].y) * (v[u].x == ref ? 1.f : exp_f(v[u].x - ref));
    }
  }
  // The shares of a row are lanes of a wave kRows apart, then waves: joined in a fixed order.
  auto join = [&](float r2, double s2) {
    if (s2 == 0.0) return;
    if (sum == 0.0) {
      ref = r2;
      sum = s2;
    } else if (r2 > ref) {
      sum = sum * exp_f(ref - r2) + s2;
      ref = r2;
    } else {
      sum += r2 == ref ? s2 : s2 * exp_f(r2 - ref);
    }
  };
#pragma unroll
  for (int o = kRows; o < 64; o <<= 1) {
    const float r2 = __shfl_xor(ref, o, 64);
    const double s2 = __shfl_xor(sum, o, 64);
    const float l2 = __shfl_xor(low, o, 64);
    const bool lower = (threadIdx.x & o) == 0;         // the same order in both lanes
    if (lower) {
      join(r2, s2);
    } else {
      const float r1 = ref;
      const double s1 = sum;
      ref = r2;
      sum = s2;
      join(r1, s1);
    }
    low = fminf(low, l2);
  }
  if ((threadIdx.x & 63) < kRows) {
    sRef[threadIdx.x >> 6][lrow] = ref;
    sLow[threadIdx.x >> 6][lrow] = low;
    sSum[threadIdx.x >> 6][lrow] = sum;
  }
  __syncthreads();
  ref = sRef[0][lrow];
  sum = sSum[0][lrow];
  low = sLow[0][lrow];
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    join(sRef[i][lrow], sSum[i][lrow]);
    low = fminf(low, sLow[i][lrow]);
  }
  const float new_ref = ref;                         // of this piece
  const float old_ref = live && !first ? h.ref[row] : -3.4e38f;
  const double old = live && !first ? h.sum[row] : 0.0;
  const float top = old == 0.0 ? new_ref : fmaxf(new_ref, old_ref);
  if (live && scale_e && low < top)
    for (int g = w; g < groups; g += kShare) {
      const float2 v = part[pitch * g];
      if (v.y == 0.f || v.x == top) continue;
      const float f = shift_of(v.x, top);
      uint4 *e = reinterpret_cast<uint4 *>(pc.E + static_cast<int64_t>(row) * pc.pitch + 64 * g);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 u = e[c];
        const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(u2f(uu[q] << 16) * f, u2f(uu[q] & 0xffff0000u) * f);
        e[c] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  __syncthreads();                                   // all threads of the row have read its state
  if (w == 0 && live) {
    const float f = old == 0.0 ? 0.f : old_ref == top ? 1.f : exp_f(old_ref - top);
    const double all = old * f + (sum == 0.0 || new_ref == top ? sum : sum * exp_f(new_ref - top));
    if (loss) {
      const RowResult r(all, h.zt[row], top);
      loss[blockIdx.x] = r.loss;
      lse[2 * blockIdx.x] = r.lse[0];
      lse[2 * blockIdx.x + 1] = r.lse[1];
    } else {
      h.ref[row] = top;
      h.sum[row] = all;
      h.factor[row] = f;
    }
  }
}

// ---------------------------------------------------------------------------
// C [split][row][K] (fp32) = factor C + sum over the split's words of E W.  6144 rows x
// 16384 words x 4096: 693 to 741 us (1.11 to 1.19 PFLOP/s).  225 rows x 50001 x 1088: 51 us in
// 32 splits of 5 tiles; 51 and 64 splits, which fill the chip, make the whole call
// slower by what their sums cost (100, 104 and 108 us), as do Mid tiles (106).
template <class S>
__global__ __launch_bounds__(S::kThreads, 2) void k_head_acc(const uint16_t *__restrict__ W, int V, int K, int v0, HeadCut cut, int first,
                                                               HeadRows h, HeadPiece pc, float *__restrict__ C) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[S::kLds];
  const int count = h.count[0];
  const int trows = (count + S::kBM - 1) / S::kBM, tcols = (K + S::kBN - 1) / S::kBN;
  const int tiles = trows * tcols;
  if (tiles == 0) return;
  const int splits = splits_for(tiles, cut);
  const int KT = pc.pitch / kBK;
  // A split after the other, so that the tiles at work share its words.
  const int split = blockIdx.x / tiles;
  int tr, tc;
  if (split >= splits || !place(blockIdx.x - split * tiles, trows, tcols, tr, tc)) return;
  const int k0 = static_cast<int>(static_cast<int64_t>(KT) * split / splits);
  const int k1 = static_cast<int>(static_cast<int64_t>(KT) * (split + 1) / splits);
  const int m0 = tr * S::kBM, c0 = tc * S::kBN;
  Acc<S> acc;
  if (k1 > k0)
    tile<S, true>(smem, pc.E + static_cast<int64_t>(kBK) * k0, pc.pitch, [&](int row) { return min(m0 + row, count - 1); },
                  W + (static_cast<int64_t>(v0) + kBK * k0) * K, K, c0, K - 1, V - 1 - v0 - kBK * k0, k1 - k0, acc);
  else
    clear<S>(acc);
  const Place<S> w;
#pragma unroll
  for (int i = 0; i < S::kFM; ++i) {
    const int row = m0 + w.row0() + 32 * i + w.lr;
    if (row >= count) continue;
    const float f = first ? 0.f : h.factor[row];
    float *c = C + (static_cast<int64_t>(split) * pc.rows + row) * K;
#pragma unroll
    for (int j = 0; j < S::kFN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = c0 + w.col0() + 32 * j + 8 * q + 4 * w.lh;
        if (k < K)
          add_to(reinterpret_cast<f32x4_t *>(c + k), f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]},
                 first, f);
      }
  }
}

// ---------------------------------------------------------------------------
// Up to kHeadSmall rows: bound by reading W, once for the logits and once more for the
// gradient, so both kernels keep three steps of it in flight in a ring of four
// stages, and the few rows of X or E go along from L2.  One row x 32000 x 4096: 57 us
// (4.6 TB/s; the tiles above took 117 and their launches the rest of 150), with the
// gradient 109 for the whole call; 64 rows with it 117.
namespace {
constexpr int kSmThreads = 256;
constexpr int kSmRing = 4;
constexpr int kSmWords = 64;      // words of a workgroup (k_head_small)
constexpr int kSmCols = 128;      // columns of a workgroup (k_head_small_acc)

template <int kMB>
constexpr int sm_row_dma() { return (2 * kMB + 3) / 4; }   // DMA instructions a wave and stage for 16 kMB rows of 128 bytes

// One stage's rows of X or E (row r of the list at off(r), 128 bytes from `col` on); surplus
// instructions repeat the last 8 rows.
template <int kMB, class Off>
__device__ __forceinline__ void sm_rows(uint32_t dst, const void *base, int wave, int lane, Off off) {
#pragma unroll
  for (int j = 0; j < sm_row_dma<kMB>(); ++j) {
    const int u = min(wave * sm_row_dma<kMB>() + j, 2 * kMB - 1);
    const int row = 8 * u + (lane >> 3);
    dma16(base, off(j) + 16 * ((lane & 7) ^ ((row & 7) ^ ((row >> 3) & 1))), __builtin_amdgcn_readfirstlane(dst + 1024 * u));
  }
}

// Waits until a step has landed while `ahead` later ones (at most 2) of kDma instructions each may be in flight.
template <int kDma>
__device__ __forceinline__ void sm_step_barrier(int ahead) {
  if (ahead >= 2)
    raw_barrier<wait_imm(2 * kDma, 0)>();
  else if (ahead == 1)
    raw_barrier<wait_imm(kDma, 0)>();
  else
    raw_barrier<wait_imm(0, 0)>();
}
}  // namespace

// k_head_rows and k_head_logits for M <= 16 kMB rows: 64 words a workgroup, 16 a
// wave, on 16 x 16 tiles (lane: row l % 16, words 4 (l / 16) + e).
template <int kMB, bool kE>
__global__ __launch_bounds__(kSmThreads) void k_head_small(const uint16_t *__restrict__ X, const int64_t *__restrict__ target, int M,
                                                           const uint16_t *__restrict__ W, int V, int K, int v0, int words, HeadRows h,
                                                           HeadPiece pc) {
  constexpr int kStage = kSmWords * 128 + kMB * 2048;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSmRing * kStage];
  __shared__ int sRow[64], sTgt[64];
  __shared__ float sTop[4][16 * kMB], sSum[4][16 * kMB];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = lane < M ? target[lane] : -1;
  const bool real = t >= 0 && t < V;
  const uint64_t mask = __ballot(real);
  const int count = __popcll(mask), rank = __popcll(mask & ((uint64_t{1} << lane) - 1));
  if (wave == 0) {
    if (real) {
      sRow[rank] = lane;
      sTgt[rank] = static_cast<int>(t);
    }
    if (blockIdx.x == 0) {
      if (real) {
        h.list[rank] = lane;
        h.tgt[rank] = static_cast<int>(t);
      }
      if (lane < M) h.place[lane] = real ? rank : -1;
      if (lane == 0) h.count[0] = count;
    }
  }
  if (count == 0) return;
  __syncthreads();
  const int w0 = blockIdx.x * kSmWords;             // of the piece
  const uint16_t *Wp = W + static_cast<int64_t>(v0 + w0) * K;
  uint32_t wo[2], xo[sm_row_dma<kMB>()];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = 8 * (2 * wave + j) + (lane >> 3);
    wo[j] = static_cast<uint32_t>(min(row, words - 1 - w0)) * K * 2 + 16 * ((lane & 7) ^ ((row & 7) ^ ((row >> 3) & 1)));
  }
#pragma unroll
  for (int j = 0; j < sm_row_dma<kMB>(); ++j) {
    const int u = min(wave * sm_row_dma<kMB>() + j, 2 * kMB - 1);
    xo[j] = static_cast<uint32_t>(sRow[min(8 * u + (lane >> 3), count - 1)]) * K * 2;
  }
  const uint32_t lds0 = lds_addr(smem);
  auto issue = [&](int kt) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + (kt & (kSmRing - 1)) * kStage;
#pragma unroll
    for (int j = 0; j < 2; ++j) dma16(Wp + 64 * kt, wo[j], __builtin_amdgcn_readfirstlane(dst + (2 * wave + j) * 1024));
    sm_rows<kMB>(dst + kSmWords * 128, X + 64 * kt, wave, lane, [&](int j) { return xo[j]; });
  };
  constexpr int kDma = 2 + sm_row_dma<kMB>();
  const int KT = K / 64;
  f32x4_t acc[kMB];
#pragma unroll
  for (int mb = 0; mb < kMB; ++mb) acc[mb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int kt = 0; kt < min(3, KT); ++kt) issue(kt);
  const int lr = lane & 15, lg = lane >> 4;
  for (int kt = 0; kt < KT; ++kt) {
    sm_step_barrier<kDma>(KT - 1 - kt);
    if (kt + 3 < KT) issue(kt + 3);
    const uint8_t *ws = smem + (kt & (kSmRing - 1)) * kStage, *xs = ws + kSmWords * 128;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bf16x8_t a = *reinterpret_cast<const bf16x8_t *>(ws + swz128(16 * wave + lr, 4 * s + lg));
#pragma unroll
      for (int mb = 0; mb < kMB; ++mb)
        acc[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, *reinterpret_cast<const bf16x8_t *>(xs + swz128(16 * mb + lr, 4 * s + lg)),
                                                          acc[mb], 0, 0, 0);
    }
  }
  const int first_word = w0 + 16 * wave + 4 * lg;    // of this lane, in the piece
#pragma unroll
  for (int mb = 0; mb < kMB; ++mb) {
    const int row = 16 * mb + lr;
    const int rel = row < count ? sTgt[row] - v0 - first_word : -1;
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (rel == e) h.zt[row] = acc[mb][e];
      if (rel == e || first_word + e >= words) acc[mb][e] = -INFINITY;
      top = fmaxf(top, acc[mb][e]);
    }
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    if (lg == 0) sTop[wave][row] = top;
  }
  __syncthreads();
#pragma unroll
  for (int mb = 0; mb < kMB; ++mb) {
    const int row = 16 * mb + lr;
    const float ref = ref_of(fmaxf(fmaxf(sTop[0][row], sTop[1][row]), fmaxf(sTop[2][row], sTop[3][row])));
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[mb][e] = exp_f(acc[mb][e] - ref);
      sum += acc[mb][e];
    }
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    if (lg == 0) sSum[wave][row] = sum;
    if constexpr (kE)
      if (row < count)
        *reinterpret_cast<uint2 *>(pc.E + static_cast<int64_t>(row) * pc.pitch + first_word) =
            make_uint2(pack_bf16x2(acc[mb][0], acc[mb][1]), pack_bf16x2(acc[mb][2], acc[mb][3]));
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < count) {
    const int row = threadIdx.x;
    const float ref = ref_of(fmaxf(fmaxf(sTop[0][row], sTop[1][row]), fmaxf(sTop[2][row], sTop[3][row])));
    pc.part[static_cast<int64_t>(blockIdx.x) * pc.rows + row] = make_float2(ref, (sSum[0][row] + sSum[1][row]) + (sSum[2][row] + sSum[3][row]));
  }
}

// k_head_acc for M <= 16 kMB rows: 128 columns a workgroup, 32 a wave, over one of
// cut.most parts of the piece's words.
template <int kMB>
__global__ __launch_bounds__(kSmThreads) void k_head_small_acc(const uint16_t *__restrict__ W, int V, int K, int v0, HeadCut cut, int first,
                                                               HeadRows h, HeadPiece pc, float *__restrict__ C) {
  constexpr int kStage = 64 * 2 * kSmCols + kMB * 2048;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSmRing * kStage];
  const int count = h.count[0];
  if (count == 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = (K + kSmCols - 1) / kSmCols;
  const int split = blockIdx.x / cols, c0 = blockIdx.x % cols * kSmCols;
  const int KT = pc.pitch / 64;
  const int k0 = static_cast<int>(static_cast<int64_t>(KT) * split / cut.most);
  const int n = static_cast<int>(static_cast<int64_t>(KT) * (split + 1) / cut.most) - k0;
  const uint16_t *Wp = W + (static_cast<int64_t>(v0) + 64 * k0) * K;
  const uint16_t *Ep = pc.E + 64 * k0;
  const int last = V - 1 - v0 - 64 * k0;             // rows of W past it are repeated: E is zero there
  // rows of 256 bytes, four a DMA instruction
  auto wrow = [&](int j) { return 4 * (4 * wave + j) + (lane >> 4); };
  uint32_t wo[4], eo[sm_row_dma<kMB>()];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = wrow(j);
    const int chunk = (lane & 15) ^ (((row & 3) << 2) | ((row >> 2) & 3));
    wo[j] = 2 * static_cast<uint32_t>(min(c0 + 8 * chunk, K - 8));
  }
#pragma unroll
  for (int j = 0; j < sm_row_dma<kMB>(); ++j) {
    const int u = min(wave * sm_row_dma<kMB>() + j, 2 * kMB - 1);
    eo[j] = static_cast<uint32_t>(min(8 * u + (lane >> 3), count - 1)) * pc.pitch * 2;
  }
  const uint32_t lds0 = lds_addr(smem);
  auto issue = [&](int kt) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + (kt & (kSmRing - 1)) * kStage;
    const uint16_t *base = Wp + static_cast<int64_t>(64) * kt * K;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      dma16(base, static_cast<uint32_t>(min(wrow(j), last - 64 * kt)) * K * 2 + wo[j],
            __builtin_amdgcn_readfirstlane(dst + (4 * wave + j) * 1024));
    sm_rows<kMB>(dst + 64 * 2 * kSmCols, Ep + 64 * kt, wave, lane, [&](int j) { return eo[j]; });
  };
  constexpr int kDma = 4 + sm_row_dma<kMB>();
  f32x4_t acc[2][kMB];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int mb = 0; mb < kMB; ++mb) acc[b][mb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int lr = lane & 15, lg = lane >> 4;
  uint32_t to[2][2];                                 // transposed reads: columns 32 wave + 16 b + l % 16, words 8 lg + 4 h .. +3
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
      to[b][hh] = static_cast<uint32_t>(
          gemm16::swz_wide<gemm16::Mid>(8 * lg + 4 * hh + (lr >> 2), 4 * wave + 2 * b + ((lr & 3) >> 1)) + 8 * (lr & 1));
  static_assert(gemm16::Mid::kBN == kSmCols, "rows of 256 bytes");
  for (int kt = 0; kt < min(3, n); ++kt) issue(kt);
  for (int kt = 0; kt < n; ++kt) {
    sm_step_barrier<kDma>(n - 1 - kt);
    if (kt + 3 < n) issue(kt + 3);
    const uint8_t *ws = smem + (kt & (kSmRing - 1)) * kStage, *es = ws + 64 * 2 * kSmCols;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8_t x[kMB];
#pragma unroll
      for (int mb = 0; mb < kMB; ++mb) x[mb] = *reinterpret_cast<const bf16x8_t *>(es + swz128(16 * mb + lr, 4 * s + lg));
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const gemm16::bf16x4_t lo = gemm16::ds_tr16(ws + to[b][0] + 64 * kSmCols * s);
        const gemm16::bf16x4_t hi = gemm16::ds_tr16(ws + to[b][1] + 64 * kSmCols * s);
        const bf16x8_t a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int mb = 0; mb < kMB; ++mb) acc[b][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, x[mb], acc[b][mb], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int mb = 0; mb < kMB; ++mb) {
    const int row = 16 * mb + lr;
    if (row >= count) continue;
    const float f = first ? 0.f : h.factor[row];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int k = c0 + 32 * wave + 16 * b + 4 * lg;
      if (k < K) add_to(reinterpret_cast<f32x4_t *>(C + (static_cast<int64_t>(split) * pc.rows + row) * K + k), acc[b][mb], first, f);
    }
  }
}

// ---------------------------------------------------------------------------
// A workgroup a row of X and 2048 columns: its loss and log-sum-exp; with kGrad 1
// (bf16) or 2 (fp32) its gradient, weight (C / sum + (p_t - 1) W_t).  Bound by reading C:
// 8192 rows x 4096, 6144 with a target, two splits: 66 to 71 us; 225 rows x 1088, 32
// splits: 12 (31 MB, eight splits' loads of a thread at once).
template <int kGrad>
__global__ __launch_bounds__(256) void k_head_finish(const uint16_t *__restrict__ W, int K, const float *__restrict__ weight, HeadRows h,
                                                     int rows, HeadCut cut, const float *__restrict__ C, float *__restrict__ loss,
                                                     float *__restrict__ lse, void *__restrict__ dX) {
  const int64_t m = blockIdx.x;
  const int at = h.place[m];
  float l = 0.f, lse0 = 0.f, lse1 = 0.f, inv = 0.f;
  if (at >= 0) {
    const RowResult r(h.sum[at], h.zt[at], h.ref[at]);
    l = r.loss;
    lse0 = r.lse[0];
    lse1 = r.lse[1];
    inv = r.inv;
  }
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    loss[m] = l;
    lse[2 * m] = lse0;
    lse[2 * m + 1] = lse1;
  }
  if constexpr (kGrad != 0) {
    const float g = at < 0 ? 0.f : (weight ? weight[m] : 1.f);
    const float pt = expm1f(-l);                     // p_t - 1
    const int splits = splits_for((h.count[0] + cut.bm - 1) / cut.bm * ((K + cut.bn - 1) / cut.bn), cut);
    const uint16_t *wt = W + static_cast<int64_t>(at < 0 ? 0 : h.tgt[at]) * K;
    const int k = 8 * (blockIdx.y * 256 + threadIdx.x);
    if (k < K) {
      float v[8] = {};
      if (at >= 0) {
        for (int s0 = 0; s0 < splits; s0 += 8) {       // 8 splits' loads at once, added in order
          f32x4_t c[8][2];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const f32x4_t *p = reinterpret_cast<const f32x4_t *>(C + (static_cast<int64_t>(min(s0 + u, splits - 1)) * rows + at) * K + k);
            c[u][0] = p[0];
            c[u][1] = p[1];
          }
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (s0 + u < splits)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[e] += c[u][0][e];
                v[4 + e] += c[u][1][e];
              }
        }
        const uint4 wv = *reinterpret_cast<const uint4 *>(wt + k);
        const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = g * (v[2 * e] * inv + pt * u2f(ww[e] << 16));
          v[2 * e + 1] = g * (v[2 * e + 1] * inv + pt * u2f(ww[e] & 0xffff0000u));
        }
      }
      if constexpr (kGrad == 1) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dX) + m * K + k) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      } else {
        f32x4_t *o = reinterpret_cast<f32x4_t *>(static_cast<float *>(dX) + m * K + k);
        o[0] = f32x4_t{v[0], v[1], v[2], v[3]};
        o[1] = f32x4_t{v[4], v[5], v[6], v[7]};
      }
    }
  }
}

// dX [M, K] = bf16(g_m D_m), 0 where D_m is that of a row without a target (its g may be anything).
__global__ __launch_bounds__(256) void k_head_scale(const float *__restrict__ D, int64_t M, int K, const int64_t *__restrict__ target, int V,
                                                    const float *__restrict__ g, uint16_t *__restrict__ dX) {
  const int64_t m = blockIdx.x;
  const int64_t t = target[m];
  const bool real = t >= 0 && t < V;
  const float f = real ? g[m] : 0.f;
  for (int k = 8 * threadIdx.x; k < K; k += 8 * 256) {
    const f32x4_t *d = reinterpret_cast<const f32x4_t *>(D + m * K + k);
    const f32x4_t a = d[0], b = d[1];
    uint4 v = make_uint4(pack_bf16x2(f * a[0], f * a[1]), pack_bf16x2(f * a[2], f * a[3]), pack_bf16x2(f * b[0], f * b[1]),
                         pack_bf16x2(f * b[2], f * b[3]));
    if (!real) v = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4 *>(dX + m * K + k) = v;
  }
}

// ---------------------------------------------------------------------------
// dz^T [word][pitch] of words v0 .. v0 + words - 1 and the listed rows, in bf16;
// zeros in the columns count .. (count filled up to 64) - 1.  The target's p_t - 1 is
// expm1(-loss) where the row's pair holds the loss (see RowResult): there p_t, from a
// logit that another order of sums rounded otherwise, says nothing of 1 - p_t.
// kTwo (up to kHeadSmall rows): a second 64 columns hold what the first lost to bf16.  A word
// that is the target of one row has that row's dz times X for its row of dW, and nothing
// averages the roundings of few rows (one row of 17000 words: error of dW against float64
// 1.3 times that of its own rounding, 1.0 so; 17000 to 131072 words, 1 to 64 rows: dW 5 to 10 % longer,
// 168 to 178 us at 64 x 32000 x 4096).  More rows: 1.15 to 1.4 times, for half the product.
// 2048 rows x 65536 words x 4096: 931 to 956 us (1.15 to 1.18 PFLOP/s), as k_head_dw below.
template <class S, bool kTwo>
__global__ __launch_bounds__(S::kThreads, 2) void k_head_dz(const uint16_t *__restrict__ Xc, const uint16_t *__restrict__ W, int K, int v0,
                                                              int words, HeadRows h, const float *__restrict__ lse,
                                                              const float *__restrict__ weight, int64_t pitch, uint16_t *__restrict__ Zt) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[S::kLds];
  __shared__ float sRef[S::kBN], sRest[S::kBN], sG[S::kBN], sOwn[S::kBN];   // sOwn: the target's p - 1, above 0 where p is to be used
  __shared__ int sT[S::kBN];
  const int count = h.count[0];
  int tr, tc;
  if (!place(blockIdx.x, (words + S::kBM - 1) / S::kBM, (count + S::kBN - 1) / S::kBN, tr, tc)) return;
  const int w0 = tr * S::kBM, c0 = tc * S::kBN;
  if (threadIdx.x < S::kBN) {
    const int at = c0 + threadIdx.x;
    const bool live = at < count;
    const int64_t m = live ? h.list[at] : 0;
    const float first = live ? lse[2 * m] : 0.f, second = live ? lse[2 * m + 1] : 0.f;
    const bool sure = first > 0.f && first < kSure;
    sRef[threadIdx.x] = sure ? second : first;
    sRest[threadIdx.x] = sure ? first : second;
    sOwn[threadIdx.x] = !sure ? 1.f : first > kNoLoss ? expm1f(-first) : 0.f;
    sG[threadIdx.x] = live ? (weight ? weight[m] : 1.f) : 0.f;
    sT[threadIdx.x] = live ? h.tgt[at] - v0 : -1;
  }
  Acc<S> acc;
  tile<S, false>(smem, W + static_cast<int64_t>(v0) * K, K, [&](int row) { return min(w0 + row, words - 1); }, Xc, K, c0, count - 1, 0,
              K / kBK, acc);
  const Place<S> w;
  const int lr = w.lr, lh = w.lh;
  const int top = count - c0;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int c = w.col0() + 32 * j + 8 * (e >> 2) + 4 * lh + (e & 3);
      const float ref = sRef[c], rest = sRest[c], g = sG[c], own = sOwn[c];
      const int t = sT[c];
#pragma unroll
      for (int i = 0; i < S::kFM; ++i) {
        const float p = exp_f((acc[i][j][e] - ref) - rest);
        acc[i][j][e] = c < top ? g * (t == w0 + w.row0() + 32 * i + lr ? (own > 0.f ? p - 1.f : own) : p) : 0.f;
      }
    }
  store_bf16<S>(acc, smem, [&](int row, int col, uint4 v) {
    if (w0 + row < words && c0 + col < (kTwo ? 64 : pitch)) *reinterpret_cast<uint4 *>(Zt + (w0 + row) * pitch + c0 + col) = v;
  });
  if constexpr (kTwo) {
#pragma unroll
    for (int i = 0; i < S::kFM; ++i)
#pragma unroll
      for (int j = 0; j < S::kFN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float held = bf16_to_f32(f32_to_bf16(acc[i][j][e]));
          acc[i][j][e] = fabsf(held) < INFINITY ? acc[i][j][e] - held : 0.f;
        }
    __builtin_amdgcn_wave_barrier();                   // the first store has read its region
    store_bf16<S>(acc, smem, [&](int row, int col, uint4 v) {
      if (w0 + row < words && c0 + col < 64) *reinterpret_cast<uint4 *>(Zt + (w0 + row) * pitch + 64 + c0 + col) = v;
    });
  }
}

// dW rows v0 .. v0 + words - 1 = dz^T X over the listed rows (twice: over both parts of dz).
template <class S>
__global__ __launch_bounds__(S::kThreads, 2) void k_head_dw(const uint16_t *__restrict__ Zt, int64_t pitch,
                                                              const uint16_t *__restrict__ Xc, int K, int v0, int words, HeadRows h,
                                                              int twice, uint16_t *__restrict__ dW) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[S::kLds];
  const int KT = (h.count[0] + kBK - 1) / kBK << twice;
  int tr, tc;
  if (!place(blockIdx.x, (words + S::kBM - 1) / S::kBM, (K + S::kBN - 1) / S::kBN, tr, tc)) return;
  const int w0 = tr * S::kBM, c0 = tc * S::kBN;
  Acc<S> acc;
  if (KT > 0)
    tile<S, true>(smem, Zt, static_cast<uint32_t>(pitch), [&](int row) { return min(w0 + row, words - 1); }, Xc, K, c0, K - 1, KT * kBK - 1,
               KT, acc);
  else
    clear<S>(acc);
  store_bf16<S>(acc, smem, [&](int row, int col, uint4 v) {
    if (w0 + row < words && c0 + col < K) *reinterpret_cast<uint4 *>(dW + static_cast<int64_t>(v0 + w0 + row) * K + c0 + col) = v;
  });
}

// ---------------------------------------------------------------------------
namespace {
template <class S>
int tiles_of(int64_t rows, int64_t cols) {
  return static_cast<int>(((rows + S::kBM - 1) / S::kBM) * ((cols + S::kBN - 1) / S::kBN));
}
using gemm16::Big;
using gemm16::Deep;
using gemm16::Mid;
}  // namespace

HeadCut head_cut(int64_t M, int64_t K, int64_t words) {
  HeadCut c;
  if (M <= kHeadSmall) {
    // one or two workgroups a compute unit, as their stages allow
    c.deep = 0;
    c.bm = c.bn = 1;
    c.slots = 0;
    c.cost = 0.f;
    const int64_t cols = (K + kSmCols - 1) / kSmCols;
    c.most = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({(M <= 32 ? 512 : 256) / cols, words / 512, 64})));
    return c;
  }
  // Splits fill the chip with either tile; 128-wide ones where Big would be half empty
  // (300 x 32000 x 4096: 280 us with Big, 317 with Mid; 100 x 32000 x 4096: 208 and 189),
  // Deep ones, as they are alone on their compute unit then (128 x 32000 x 4096: 160 us
  // with Mid and 512 slots, 151 with Deep and 256).
  c.deep = M <= Deep::kBM ? 1 : 0;
  c.bm = c.deep ? Deep::kBM : Big::kBM;
  c.bn = c.deep ? Deep::kBN : Big::kBN;
  c.slots = 256;
  // a tile's 4 bytes an element out and in at 5 TB/s, against a step of 64 words of a round: 1.7 us (Deep 0.85)
  c.cost = static_cast<float>(c.bm * c.bn * 8 / 5e6) / ((c.deep ? 0.85f : 1.7f) * static_cast<float>((words + 63) / 64));
  // each at least 8 steps of 64 words long, their sums within 512 MB
  c.most = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({32, words / 512, (int64_t{1} << 27) / (M * K)})));
  return c;
}

hipError_t launch_head_rows(const int64_t *target, int M, int V, const HeadRows &h, hipStream_t s) {
  hipLaunchKernelGGL(k_head_rows, dim3(1), dim3(1024), 0, s, target, M, V, h);
  return hipGetLastError();
}

hipError_t launch_head_gather(const uint16_t *X, int M, int K, const HeadRows &h, uint16_t *Xc, hipStream_t s) {
  const int64_t n = (static_cast<int64_t>(M) + 63) / 64 * 64 * K / 8;
  hipLaunchKernelGGL(k_head_gather, dim3(static_cast<int>(std::min<int64_t>(2048, (n + 255) / 256))), dim3(256), 0, s, X, K, h,
                     M <= kHeadSmall ? 1 : 0, Xc);
  return hipGetLastError();
}

// 128 x 32000 x 4096: the loss alone takes 81.5 us with Mid tiles and 74 with Deep ones, with
// the gradient 151 and 138.
template <bool kE>
static hipError_t launch_head_logits(const uint16_t *X, int M, const uint16_t *W, int K, int v0, int words, const HeadRows &h,
                                     const HeadPiece &pc, hipStream_t s) {
  if (!gemm16::use_mid(M, words))
    hipLaunchKernelGGL((k_head_logits<Big, kE>), dim3(tiles_of<Big>(M, words)), dim3(Big::kThreads), 0, s, X, W, K, v0, words, h, pc);
  else if (gemm16::use_deep(M, words))
    hipLaunchKernelGGL((k_head_logits<Deep, kE>), dim3(tiles_of<Deep>(M, words)), dim3(Deep::kThreads), 0, s, X, W, K, v0, words, h, pc);
  else
    hipLaunchKernelGGL((k_head_logits<Mid, kE>), dim3(tiles_of<Mid>(M, words)), dim3(Mid::kThreads), 0, s, X, W, K, v0, words, h, pc);
  return hipGetLastError();
}

template <int kMB>
static hipError_t launch_head_small(const uint16_t *X, const int64_t *target, int M, const uint16_t *W, int V, int K, int v0, int words,
                                    bool first, const HeadRows &h, const HeadPiece &pc, const HeadCut &cut, float *C, float *loss, float *lse,
                                    hipStream_t s) {
  const dim3 g((words + kSmWords - 1) / kSmWords), t(kSmThreads);
  if (C)
    hipLaunchKernelGGL((k_head_small<kMB, true>), g, t, 0, s, X, target, M, W, V, K, v0, words, h, pc);
  else
    hipLaunchKernelGGL((k_head_small<kMB, false>), g, t, 0, s, X, target, M, W, V, K, v0, words, h, pc);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_head_refs<1>, dim3(M), dim3(256), 0, s, h, pc, (words + 63) / 64, first ? 1 : 0, C ? 1 : 0, loss, lse);
  e = hipGetLastError();
  if (e != hipSuccess || !C) return e;
  hipLaunchKernelGGL(k_head_small_acc<kMB>, dim3((K + kSmCols - 1) / kSmCols * cut.most), t, 0, s, W, V, K, v0, cut, first ? 1 : 0, h, pc, C);
  return hipGetLastError();
}

hipError_t launch_head_small_piece(const uint16_t *X, const int64_t *target, int M, const uint16_t *W, int V, int K, int v0, int words,
                                   bool first, const HeadRows &h, const HeadPiece &pc, const HeadCut &cut, float *C, float *loss, float *lse,
                                   hipStream_t s) {
  switch ((M + 15) / 16) {
    case 1: return launch_head_small<1>(X, target, M, W, V, K, v0, words, first, h, pc, cut, C, loss, lse, s);
    case 2: return launch_head_small<2>(X, target, M, W, V, K, v0, words, first, h, pc, cut, C, loss, lse, s);
    case 3: return launch_head_small<3>(X, target, M, W, V, K, v0, words, first, h, pc, cut, C, loss, lse, s);
    default: return launch_head_small<4>(X, target, M, W, V, K, v0, words, first, h, pc, cut, C, loss, lse, s);
  }
}

hipError_t launch_head_piece(const uint16_t *X, int M, const uint16_t *W, int V, int K, int v0, int words, bool first, const HeadRows &h,
                             const HeadPiece &pc, const HeadCut &cut, float *C, hipStream_t s) {
  hipError_t e = C ? launch_head_logits<true>(X, M, W, K, v0, words, h, pc, s) : launch_head_logits<false>(X, M, W, K, v0, words, h, pc, s);
  if (e != hipSuccess) return e;
  // more threads a row while the rows are few (300 rows, 782 groups: 13 us with 16 threads a row)
  if (M <= 2048)
    hipLaunchKernelGGL(k_head_refs<4>, dim3((M + 3) / 4), dim3(256), 0, s, h, pc, (words + 63) / 64, first ? 1 : 0, C ? 1 : 0,
                       nullptr, nullptr);
  else
    hipLaunchKernelGGL(k_head_refs<16>, dim3((M + 15) / 16), dim3(256), 0, s, h, pc, (words + 63) / 64, first ? 1 : 0, C ? 1 : 0,
                       nullptr, nullptr);
  e = hipGetLastError();
  if (e != hipSuccess || !C) return e;
  // workgroups for any number of rows that have a target
  const int trows = (M + cut.bm - 1) / cut.bm, tcols = (K + cut.bn - 1) / cut.bn;
  int items = trows * tcols;
  for (int r = 1; r <= trows && r * tcols <= 50 * cut.slots; ++r) items = std::max(items, r * tcols * splits_for(r * tcols, cut));
  const dim3 grid(items);
  if (cut.deep)
    hipLaunchKernelGGL(k_head_acc<Deep>, grid, dim3(Deep::kThreads), 0, s, W, V, K, v0, cut, first ? 1 : 0, h,
                       pc, C);
  else
    hipLaunchKernelGGL(k_head_acc<Big>, grid, dim3(Big::kThreads), 0, s, W, V, K, v0, cut, first ? 1 : 0, h,
                       pc, C);
  return hipGetLastError();
}

hipError_t launch_head_finish(const uint16_t *W, int64_t M, int K, const float *weight, const HeadRows &h, const HeadCut &cut, const float *C,
                              float *loss, float *lse, void *dX, int grad, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(M), grad ? (K + 2047) / 2048 : 1), t(grad ? 256 : 64);
  const int rows = static_cast<int>(M);
  if (grad == 0)
    hipLaunchKernelGGL(k_head_finish<0>, g, t, 0, s, W, K, weight, h, rows, cut, C, loss, lse, dX);
  else if (grad == 1)
    hipLaunchKernelGGL(k_head_finish<1>, g, t, 0, s, W, K, weight, h, rows, cut, C, loss, lse, dX);
  else
    hipLaunchKernelGGL(k_head_finish<2>, g, t, 0, s, W, K, weight, h, rows, cut, C, loss, lse, dX);
  return hipGetLastError();
}

hipError_t launch_head_scale(const float *D, int64_t M, int K, const int64_t *target, int V, const float *g, uint16_t *dX, hipStream_t s) {
  hipLaunchKernelGGL(k_head_scale, dim3(static_cast<unsigned>(M)), dim3(256), 0, s, D, M, K, target, V, g, dX);
  return hipGetLastError();
}

hipError_t launch_head_dw(const uint16_t *Xc, int M, const uint16_t *W, int K, int v0, int words, const HeadRows &h, const float *lse,
                          const float *weight, uint16_t *Zt, uint16_t *dW, hipStream_t s) {
  const int64_t pitch = head_dw_depth(M);
  const int twice = M <= kHeadSmall ? 1 : 0;
  if (twice)   // one column of tiles of either shape
    hipLaunchKernelGGL((k_head_dz<Mid, true>), dim3(tiles_of<Mid>(words, M)), dim3(Mid::kThreads), 0, s, Xc, W, K, v0, words, h, lse,
                       weight, pitch, Zt);
  else if (gemm16::use_mid(words, M))
    hipLaunchKernelGGL((k_head_dz<Mid, false>), dim3(tiles_of<Mid>(words, M)), dim3(Mid::kThreads), 0, s, Xc, W, K, v0, words, h, lse, weight, pitch,
                       Zt);
  else
    hipLaunchKernelGGL((k_head_dz<Big, false>), dim3(tiles_of<Big>(words, M)), dim3(Big::kThreads), 0, s, Xc, W, K, v0, words, h, lse, weight, pitch,
                       Zt);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (gemm16::use_mid(words, K))
    hipLaunchKernelGGL(k_head_dw<Mid>, dim3(tiles_of<Mid>(words, K)), dim3(Mid::kThreads), 0, s, Zt, pitch, Xc, K, v0, words, h, twice, dW);
  else
    hipLaunchKernelGGL(k_head_dw<Big>, dim3(tiles_of<Big>(words, K)), dim3(Big::kThreads), 0, s, Zt, pitch, Xc, K, v0, words, h, twice, dW);
  return hipGetLastError();
}

}  // namespace qlora
