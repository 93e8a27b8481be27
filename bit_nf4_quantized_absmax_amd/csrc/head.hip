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
//  * ref is a multiple of 32 near the largest logit of a row's 64 words (within
//    16 of it), so that almost always the words of a row, and its pieces, have the same: e^16
//    and what lies 71 below the largest fit into fp32 and bf16 alike, whose
//    relative precision does not depend on the scale.  Where they differ, the sums (k_head_refs)
//    and E (there too) are brought to the largest, and the gradient so far by
//    the next product's epilogue.
//  * The target's own term is left out of E and of the sums, and joins them in 64
//    bits at the end (k_head_finish): the loss is log(1 + sum / e^(z_t - ref)), and
//    (p_t - 1) W_t is added in fp32, where a rounded p_t near 1 would lose both.  E's rounding to bf16 is
//    the operand type of the second product; its error is that of one output rounding, averaged over words.
//  * Rows without a target take no part: the rows that have one are listed
//    first (k_head_rows) and copied together (k_head_gather).
//  * dW, where the head is tuned as well, makes its logits a second time, for
//    dz needs the whole row's sum: dz^T piece by piece in bf16 (k_head_dz), then
//    dz^T X (k_head_dw).
#include <algorithm>

#include "common.h"
#include "gemm16.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kBucket = 32.f;

// e^x through the hardware's 2^x (x <= 16 here; what underflows is 0).
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// The reference of words whose largest logit is top; 0 where that is no number.
__device__ __forceinline__ float ref_of(float top) {
  const float r = kBucket * rintf(top * (1.f / kBucket));
  return fabsf(top) <= 3.0e38f ? r : 0.f;
}

__device__ __forceinline__ float swap_halves(float v) { return __shfl_xor(v, 32, 64); }

}  // namespace

// ---------------------------------------------------------------------------
// Rows with a target, in order: list [count] of row numbers, tgt [count], place
// [M] of a row in the list (-1: none).  One workgroup.
__global__ __launch_bounds__(1024) void k_head_rows(const int64_t *__restrict__ target, int M, int V, HeadRows h) {
  __shared__ int wsum[16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int base = 0;
  for (int64_t m0 = 0; m0 < M; m0 += 1024) {
    const int64_t m = m0 + threadIdx.x;
    const int64_t t = m < M ? target[m] : -1;
    const bool real = t >= 0 && t < V;
    const uint64_t mask = __ballot(real);
    if (lane == 0) wsum[wave] = __popcll(mask);
    __syncthreads();
    int before = base, all = 0;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) before += wsum[w];
      all += wsum[w];
    }
    const int at = before + static_cast<int>(__popcll(mask & ((uint64_t{1} << lane) - 1)));
    if (m < M) h.place[m] = real ? at : -1;
    if (real) {
      h.list[at] = static_cast<int>(m);
      h.tgt[at] = static_cast<int>(t);
    }
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) h.count[0] = base;
}

// Xc [count filled up to 64][K]: the listed rows of X, zeros behind.
__global__ __launch_bounds__(256) void k_head_gather(const uint16_t *__restrict__ X, int K, HeadRows h, uint16_t *__restrict__ Xc) {
  const int count = h.count[0], rows = (count + 63) / 64 * 64, per = K >> 3;
  const int64_t all = static_cast<int64_t>(rows) * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int row = static_cast<int>(i / per), c = static_cast<int>(i % per);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < count) v = *reinterpret_cast<const uint4 *>(X + static_cast<int64_t>(h.list[row]) * K + 8 * c);
    *reinterpret_cast<uint4 *>(Xc + static_cast<int64_t>(row) * K + 8 * c) = v;
  }
}

// ---------------------------------------------------------------------------
// Words v0 .. v0 + words - 1 of the listed rows: part [64-word group][row] =
// (ref, sum of e^(z - ref)) without the target, the target's logit where it is
// among them, and with kE the matrix E [row][pitch], pitch = words filled up to 64,
// zero there and at the target.
template <bool kE>
__global__ __launch_bounds__(gemm16::kThreads) void k_head_logits(const uint16_t *__restrict__ Xc, const uint16_t *__restrict__ W, int K,
                                                                  int v0, int words, HeadRows h, HeadPiece pc) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
  const int count = h.count[0];
  int tr, tc;
  if (!place(blockIdx.x, (count + kBM - 1) / kBM, (words + kBN - 1) / kBN, tr, tc)) return;
  const int m0 = tr * kBM, c0 = tc * kBN;
  f32x16_t acc[4][2];
  tile<false>(smem, Xc, K, [&](int row) { return min(m0 + row, count - 1); }, W + static_cast<int64_t>(v0) * K, K, c0, words - 1, 0,
              K / kBK, acc);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3, lr = lane & 31, lh = lane >> 5;
  const int cw = c0 + 64 * wn;                       // first word (of the piece) of this wave
  const bool edge = cw + 64 > words;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = m0 + 128 * wm + 32 * i + lr;
    const bool live = row < count;
    const int rel = live ? h.tgt[row] - v0 - cw - 4 * lh : -1;   // of this half's words: 0 .. 3, 8 .. 11, ...
    if (edge) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (cw + 32 * j + 8 * (e >> 2) + 4 * lh + (e & 3) >= words) acc[i][j][e] = -INFINITY;
    }
    float top = acc[i][0][0];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][j][e]);
    top = fmaxf(top, swap_halves(top));
    const float ref = ref_of(top);
    float sum = 0.f;
    const bool hit = rel >= 0 && rel < 64 && (rel & 4) == 0;
    const bool any = __ballot(hit) != 0;
    float zt = 0.f;
    if (any) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (rel == 32 * j + 8 * (e >> 2) + (e & 3)) zt = acc[i][j][e];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = exp_f(acc[i][j][e] - ref);
        sum += x;
        acc[i][j][e] = x;
      }
    if (any) {                                       // again without the target
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (rel == 32 * j + 8 * (e >> 2) + (e & 3)) acc[i][j][e] = 0.f;
          sum += acc[i][j][e];
        }
    }
    sum += swap_halves(sum);
    if (live && hit) h.zt[row] = zt;
    if (live && lh == 0 && cw < words) pc.part[static_cast<int64_t>(cw >> 6) * pc.rows + row] = make_float2(ref, sum);
  }
  if constexpr (kE)
    store_bf16(acc, smem, [&](int row, int col, uint4 v) {
      if (m0 + row < count && c0 + col < pc.pitch)
        *reinterpret_cast<uint4 *>(pc.E + static_cast<int64_t>(m0 + row) * pc.pitch + c0 + col) = v;
    });
}

// ---------------------------------------------------------------------------
// A row's sum with this piece's groups, at the largest of their references and
// its own so far: state [row] = (ref, sum), factor [row] = e^(old ref - ref) for
// the gradient so far (0 at the first piece).  Groups of E at a smaller reference are
// brought to this one.  Workgroup: 64 rows, 4 waves share the groups.
__global__ __launch_bounds__(256) void k_head_refs(HeadRows h, HeadPiece pc, int groups, int first, int scale_e) {
  __shared__ float top[4][64];
  __shared__ double sums[4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int row = blockIdx.x * 64 + lane, count = h.count[0];
  const bool live = row < count;
  const float2 *part = pc.part + row;
  float ref = -3.4e38f;
  if (live)
    for (int g = w; g < groups; g += 4) {
      const float2 v = part[static_cast<int64_t>(g) * pc.rows];
      if (v.y != 0.f) ref = fmaxf(ref, v.x);
    }
  top[w][lane] = ref;
  __syncthreads();
  ref = fmaxf(fmaxf(top[0][lane], top[1][lane]), fmaxf(top[2][lane], top[3][lane]));
  float old_ref = -3.4e38f;
  double old = 0.0;
  if (live && !first) {
    old_ref = h.ref[row];
    old = h.sum[row];
  }
  ref = fmaxf(ref, old_ref);
  double sum = 0.0;
  if (live)
    for (int g = w; g < groups; g += 4) {
      const float2 v = part[static_cast<int64_t>(g) * pc.rows];
      if (v.y == 0.f) continue;
      const float f = v.x == ref ? 1.f : exp_f(v.x - ref);
      sum += static_cast<double>(v.y) * f;
      if (scale_e && f != 1.f) {
        uint16_t *e = pc.E + static_cast<int64_t>(row) * pc.pitch + 64 * g;
        for (int c = 0; c < 64; c += 2) {
          const uint32_t u = *reinterpret_cast<uint32_t *>(e + c);
          *reinterpret_cast<uint32_t *>(e + c) = pack_bf16x2(u2f(u << 16) * f, u2f(u & 0xffff0000u) * f);
        }
      }
    }
  sums[w][lane] = sum;
  __syncthreads();
  if (w == 0 && live) {
    const float f = old_ref == ref ? 1.f : (old == 0.0 ? 0.f : exp_f(old_ref - ref));
    h.ref[row] = ref;
    h.sum[row] = old * f + (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
    h.factor[row] = first ? 0.f : f;
  }
}

// ---------------------------------------------------------------------------
// C [split][row][K] (fp32) = factor C + sum over the split's words of E W.
__global__ __launch_bounds__(gemm16::kThreads) void k_head_acc(const uint16_t *__restrict__ W, int V, int K, int v0, int splits, int first,
                                                               HeadRows h, HeadPiece pc, float *__restrict__ C) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
  const int count = h.count[0];
  const int trows = (count + kBM - 1) / kBM, tcols = (K + kBN - 1) / kBN;
  // splits of one tile are apart by a multiple of the tiles, so that an XCD's tiles share a split's words
  int tr, tc;
  const int tiles = trows * tcols;
  if (tiles == 0) return;
  const int split = blockIdx.x / tiles;
  if (split >= splits || !place(blockIdx.x - split * tiles, trows, tcols, tr, tc)) return;
  const int KT = pc.pitch / kBK;
  const int k0 = static_cast<int>(static_cast<int64_t>(KT) * split / splits);
  const int k1 = static_cast<int>(static_cast<int64_t>(KT) * (split + 1) / splits);
  const int m0 = tr * kBM, c0 = tc * kBN;
  f32x16_t acc[4][2];
  if (k1 > k0)
    tile<true>(smem, pc.E + static_cast<int64_t>(kBK) * k0, pc.pitch, [&](int row) { return min(m0 + row, count - 1); },
               W + (static_cast<int64_t>(v0) + kBK * k0) * K, K, c0, K - 1, V - 1 - v0 - kBK * k0, k1 - k0, acc);
  else
    clear(acc);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3, lr = lane & 31, lh = lane >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = m0 + 128 * wm + 32 * i + lr;
    if (row >= count) continue;
    const float f = first ? 0.f : h.factor[row];
    float *c = C + (static_cast<int64_t>(split) * pc.rows + row) * K;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = c0 + 64 * wn + 32 * j + 8 * q + 4 * lh;
        if (k >= K) continue;
        f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        f32x4_t *at = reinterpret_cast<f32x4_t *>(c + k);
        if (!first) {
          const f32x4_t o = *at;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += f * o[e];
        }
        *at = v;
      }
  }
}

// ---------------------------------------------------------------------------
// One workgroup a row of X: its loss and (ref, log sum); with kGrad 1 (bf16) or 2
// (fp32) its gradient, weight (C / sum + (p_t - 1) W_t).
template <int kGrad>
__global__ __launch_bounds__(256) void k_head_finish(const uint16_t *__restrict__ W, int K, const float *__restrict__ weight, HeadRows h,
                                                     int rows, int splits, const float *__restrict__ C, float *__restrict__ loss,
                                                     float *__restrict__ lse, void *__restrict__ dX) {
  const int64_t m = blockIdx.x;
  const int at = h.place[m];
  float l = 0.f, lg = 0.f, ref = 0.f, inv = 0.f;
  if (at >= 0) {
    const double s = h.sum[at], zt = h.zt[at];      // all words but the target, at ref; 0: there are none
    ref = h.ref[at];
    const double u = static_cast<double>(ref) - zt;
    double loss64 = s == 0.0 ? 0.0 : u > 0.0 ? u + log(s + exp(-u)) : log1p(s * exp(u));
    if (!(fabs(zt) < INFINITY) || !(s < INFINITY)) loss64 = NAN;
    inv = s == 0.0 ? 0.f : static_cast<float>(exp(-(loss64 - u)));   // loss - u = log of the whole sum at ref
    if (s == 0.0 || zt > ref + kBucket) ref = ref_of(static_cast<float>(zt));
    lg = static_cast<float>(loss64 + (zt - ref));
    l = static_cast<float>(loss64);
  }
  if (threadIdx.x == 0) {
    loss[m] = l;
    lse[2 * m] = ref;
    lse[2 * m + 1] = lg;
  }
  if constexpr (kGrad != 0) {
    const float g = at < 0 ? 0.f : (weight ? weight[m] : 1.f);
    const float pt = expm1f(-l);                     // p_t - 1
    const uint16_t *wt = W + static_cast<int64_t>(at < 0 ? 0 : h.tgt[at]) * K;
    for (int k = 8 * threadIdx.x; k < K; k += 8 * 256) {
      float v[8] = {};
      if (at >= 0) {
        for (int s = 0; s < splits; ++s) {
          const f32x4_t *c = reinterpret_cast<const f32x4_t *>(C + (static_cast<int64_t>(s) * rows + at) * K + k);
          const f32x4_t c0 = c[0], c1 = c[1];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] += c0[e];
            v[4 + e] += c1[e];
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
// zeros in the columns count .. (count filled up to 64) - 1.
__global__ __launch_bounds__(gemm16::kThreads) void k_head_dz(const uint16_t *__restrict__ Xc, const uint16_t *__restrict__ W, int K, int v0,
                                                              int words, HeadRows h, const float *__restrict__ lse,
                                                              const float *__restrict__ weight, int64_t pitch, uint16_t *__restrict__ Zt) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
  __shared__ float sRef[kBN], sRest[kBN], sG[kBN];
  __shared__ int sT[kBN];
  const int count = h.count[0];
  int tr, tc;
  if (!place(blockIdx.x, (words + kBM - 1) / kBM, (count + kBN - 1) / kBN, tr, tc)) return;
  const int w0 = tr * kBM, c0 = tc * kBN;
  if (threadIdx.x < kBN) {
    const int at = c0 + threadIdx.x;
    const bool live = at < count;
    const int64_t m = live ? h.list[at] : 0;
    sRef[threadIdx.x] = live ? lse[2 * m] : 0.f;
    sRest[threadIdx.x] = live ? lse[2 * m + 1] : 0.f;
    sG[threadIdx.x] = live ? (weight ? weight[m] : 1.f) : 0.f;
    sT[threadIdx.x] = live ? h.tgt[at] - v0 : -1;
  }
  f32x16_t acc[4][2];
  tile<false>(smem, W + static_cast<int64_t>(v0) * K, K, [&](int row) { return min(w0 + row, words - 1); }, Xc, K, c0, count - 1, 0,
              K / kBK, acc);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3, lr = lane & 31, lh = lane >> 5;
  const int top = count - c0;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int c = 64 * wn + 32 * j + 8 * (e >> 2) + 4 * lh + (e & 3);
      const float ref = sRef[c], rest = sRest[c], g = sG[c];
      const int t = sT[c];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = exp_f((acc[i][j][e] - ref) - rest);
        acc[i][j][e] = c < top ? g * (t == w0 + 128 * wm + 32 * i + lr ? p - 1.f : p) : 0.f;
      }
    }
  store_bf16(acc, smem, [&](int row, int col, uint4 v) {
    if (w0 + row < words && c0 + col < pitch) *reinterpret_cast<uint4 *>(Zt + (w0 + row) * pitch + c0 + col) = v;
  });
}

// dW rows v0 .. v0 + words - 1 = dz^T X over the listed rows.
__global__ __launch_bounds__(gemm16::kThreads) void k_head_dw(const uint16_t *__restrict__ Zt, int64_t pitch,
                                                              const uint16_t *__restrict__ Xc, int K, int v0, int words, HeadRows h,
                                                              uint16_t *__restrict__ dW) {
  using namespace gemm16;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
  const int KT = (h.count[0] + kBK - 1) / kBK;
  int tr, tc;
  if (!place(blockIdx.x, (words + kBM - 1) / kBM, (K + kBN - 1) / kBN, tr, tc)) return;
  const int w0 = tr * kBM, c0 = tc * kBN;
  f32x16_t acc[4][2];
  if (KT > 0)
    tile<true>(smem, Zt, static_cast<uint32_t>(pitch), [&](int row) { return min(w0 + row, words - 1); }, Xc, K, c0, K - 1, KT * kBK - 1,
               KT, acc);
  else
    clear(acc);
  store_bf16(acc, smem, [&](int row, int col, uint4 v) {
    if (w0 + row < words && c0 + col < K) *reinterpret_cast<uint4 *>(dW + static_cast<int64_t>(v0 + w0 + row) * K + c0 + col) = v;
  });
}

// ---------------------------------------------------------------------------
namespace {
int tiles_of(int64_t rows, int64_t cols) {
  return static_cast<int>(((rows + gemm16::kBM - 1) / gemm16::kBM) * ((cols + gemm16::kBN - 1) / gemm16::kBN));
}
}  // namespace

hipError_t launch_head_rows(const int64_t *target, int M, int V, const HeadRows &h, hipStream_t s) {
  hipLaunchKernelGGL(k_head_rows, dim3(1), dim3(1024), 0, s, target, M, V, h);
  return hipGetLastError();
}

hipError_t launch_head_gather(const uint16_t *X, int M, int K, const HeadRows &h, uint16_t *Xc, hipStream_t s) {
  const int64_t n = (static_cast<int64_t>(M) + 63) / 64 * 64 * K / 8;
  hipLaunchKernelGGL(k_head_gather, dim3(static_cast<int>(std::min<int64_t>(2048, (n + 255) / 256))), dim3(256), 0, s, X, K, h, Xc);
  return hipGetLastError();
}

hipError_t launch_head_piece(const uint16_t *Xc, int M, const uint16_t *W, int V, int K, int v0, int words, bool first, const HeadRows &h,
                             const HeadPiece &pc, int splits, float *C, hipStream_t s) {
  const int tiles = tiles_of(M, words);
  if (C)
    hipLaunchKernelGGL(k_head_logits<true>, dim3(tiles), dim3(gemm16::kThreads), 0, s, Xc, W, K, v0, words, h, pc);
  else
    hipLaunchKernelGGL(k_head_logits<false>, dim3(tiles), dim3(gemm16::kThreads), 0, s, Xc, W, K, v0, words, h, pc);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_head_refs, dim3((M + 63) / 64), dim3(256), 0, s, h, pc, (words + 63) / 64, first ? 1 : 0, C ? 1 : 0);
  e = hipGetLastError();
  if (e != hipSuccess || !C) return e;
  hipLaunchKernelGGL(k_head_acc, dim3(tiles_of(M, K) * splits), dim3(gemm16::kThreads), 0, s, W, V, K, v0, splits, first ? 1 : 0, h, pc, C);
  return hipGetLastError();
}

hipError_t launch_head_finish(const uint16_t *W, int64_t M, int K, const float *weight, const HeadRows &h, int splits, const float *C,
                              float *loss, float *lse, void *dX, int grad, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(M)), t(grad ? 256 : 64);
  const int rows = static_cast<int>(M);
  if (grad == 0)
    hipLaunchKernelGGL(k_head_finish<0>, g, t, 0, s, W, K, weight, h, rows, splits, C, loss, lse, dX);
  else if (grad == 1)
    hipLaunchKernelGGL(k_head_finish<1>, g, t, 0, s, W, K, weight, h, rows, splits, C, loss, lse, dX);
  else
    hipLaunchKernelGGL(k_head_finish<2>, g, t, 0, s, W, K, weight, h, rows, splits, C, loss, lse, dX);
  return hipGetLastError();
}

hipError_t launch_head_scale(const float *D, int64_t M, int K, const int64_t *target, int V, const float *g, uint16_t *dX, hipStream_t s) {
  hipLaunchKernelGGL(k_head_scale, dim3(static_cast<unsigned>(M)), dim3(256), 0, s, D, M, K, target, V, g, dX);
  return hipGetLastError();
}

hipError_t launch_head_dw(const uint16_t *Xc, int M, const uint16_t *W, int K, int v0, int words, const HeadRows &h, const float *lse,
                          const float *weight, uint16_t *Zt, uint16_t *dW, hipStream_t s) {
  const int64_t pitch = (static_cast<int64_t>(M) + 63) / 64 * 64;
  hipLaunchKernelGGL(k_head_dz, dim3(tiles_of(words, M)), dim3(gemm16::kThreads), 0, s, Xc, W, K, v0, words, h, lse, weight, pitch, Zt);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_head_dw, dim3(tiles_of(words, K)), dim3(gemm16::kThreads), 0, s, Zt, pitch, Xc, K, v0, words, h, dW);
  return hipGetLastError();
}

}  // namespace qlora
