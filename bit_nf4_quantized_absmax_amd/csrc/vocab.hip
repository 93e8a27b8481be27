// Losses over the vocabulary: rows of logits z [V] and p = softmax(z / tau).
//
//   log probability   lp = z_t - lse,  lse = log sum_j e^z_j
//   entropy           H  = -sum_j p_j log p_j
//   alternatives      the k largest z, the lower index first among equals
//     backward        dz_j = g_lp ([j = t] - p_j) - g_H p_j (log p_j + H)
//   distillation      q = softmax(t / tau) over the row's listed words,
//                     loss = sum_i q_i (log q_i - log p_idx(i))
//     backward        dz_j = w (p_j - sum of the q_i listed for j) / tau
//
// A slice of a row keeps its maximum a and, with e_j = 2^t_j, t_j = (z_j - a)
// log2(e) / tau, the sums s of e_j and u of e_j t_j (fp32); slices are joined
// in 64 bits:
//     s = sum f_i s_i,  u = sum f_i (u_i + d_i s_i),  f_i = 2^d_i, d_i = (a_i - a) log2(e) / tau
//     H = ln 2 (log2 s - u / s)
// log2 s >= 0 >= u: nothing cancels in H.  The log-sum-exp stays a pair (a,
// log s) whose sum it is: log p_j = (z_j - a) / tau - log s keeps its digits
// where the rounding of the sum would lose them (rows masked by a type's
// lowest value throughout: a = -3e38, p = 1 / V).
//
// Masked words are -inf: e = 0, and in u the factor is held at -300 (0 * -300
// = 0 where 0 * -inf were NaN).  A row that is all -inf has a = -inf and s =
// 0; its gradients are 0.  A NaN or +inf in a row makes its sums NaN.
//
// Rows are cut into slices of at most 16384 words (32 KB to 64 KB); a
// workgroup holds a slice in registers, so that z is read once for the
// maximum, the sums and the alternatives.  A second kernel joins a row's
// slices.  The order of every sum is fixed.
#include <math.h>

#include <algorithm>

#include "common.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr int kVThreads = 256;
constexpr int kVWaves = kVThreads / 64;
constexpr int kCandMax = 1024;          // alternatives considered by a slice
constexpr float kLog2e = 1.44269502f;   // fp32 nearest to log2(e)
constexpr int64_t kSliceMin = 2048;     // words of a slice, when there are few rows
constexpr int64_t kSliceMax = 16384;

template <typename T>
struct Words {
  static constexpr int n = 16 / static_cast<int>(sizeof(T));   // words of a 16-byte load
};

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__bf16 v) { return static_cast<float>(v); }
__device__ __forceinline__ float as_f32(_Float16 v) { return static_cast<float>(v); }

template <typename T>
struct alignas(16) Vec {
  T w[Words<T>::n];
};

// Row m of a matrix cut at 16-byte boundaries: vector v covers words v n -
// mis .. of the row, mis = the row's first word within its 16 bytes.
template <typename T>
struct Row {
  const T *p;
  int V;
  int mis;
  __device__ __forceinline__ Row(const T *base, int64_t ld, int64_t m, int v) : p(base + m * ld), V(v) {
    mis = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
  }
  __device__ __forceinline__ int first(int v) const { return v * Words<T>::n - mis; }
  // Words outside the row are -inf; only words of the row are read.
  __device__ __forceinline__ Vec<T> load(int v) const {
    const int j = first(v);
    Vec<T> x;
    if (j >= 0 && j + Words<T>::n <= V) {
      x = *reinterpret_cast<const Vec<T> *>(p + j);
    } else {
#pragma unroll
      for (int e = 0; e < Words<T>::n; ++e)
        x.w[e] = (j + e >= 0 && j + e < V) ? p[j + e] : static_cast<T>(-INFINITY);
    }
    return x;
  }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Maximum over the workgroup (every thread gets it); sh: one float a wave.
// A NaN is passed over here; it makes the sums NaN.
__device__ __forceinline__ float block_max(float v, float *sh) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  float m = sh[0];
  for (int w = 1; w < static_cast<int>(blockDim.x >> 6); ++w) m = fmaxf(m, sh[w]);
  return m;
}
__device__ __forceinline__ float block_sum(float v, float *sh) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  float m = sh[0];
  for (int w = 1; w < static_cast<int>(blockDim.x >> 6); ++w) m += sh[w];
  return m;
}

// Order-preserving integer of a float (-0 as +0; a NaN above or below all).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// A word as a key: larger for a larger logit, then for a lower index.
__device__ __forceinline__ uint64_t word_key(float v, uint32_t j) {
  return (static_cast<uint64_t>(ordered(v)) << 32) | (0xFFFFFFFFu - j);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return 0xFFFFFFFFu - static_cast<uint32_t>(k); }

struct Partial {
  float a, s, u;
};

// Slices of a launch and the workspace they leave: partials [M][S], then the
// alternatives' keys [M][S][top].
struct Slices {
  int S;             // slices of a row
  int per;           // 16-byte vectors of a slice
};

Slices slices_of(int64_t M, int64_t V, int type) {
  const int n = type == 0 ? 4 : 8;
  // enough slices for two workgroups a CU, none below kSliceMin or above kSliceMax words
  const int64_t most = (V + kSliceMin - 1) / kSliceMin, least = (V + n + kSliceMax - 1) / kSliceMax;
  const int64_t want = (512 + M - 1) / std::max<int64_t>(M, 1);
  const int64_t S = std::max(least, std::min(most, want));
  const int64_t nv = (V + 2 * n - 2) / n;   // a row that starts inside 16 bytes touches one vector more
  return Slices{static_cast<int>(S), static_cast<int>((nv + S - 1) / S)};
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t vocab_ws_bytes(int64_t M, int64_t V, int type, int top) {
  const Slices sl = slices_of(M, V, type);
  return up256(static_cast<size_t>(M) * sl.S * sizeof(Partial)) + static_cast<size_t>(M) * sl.S * top * sizeof(uint64_t);
}

// One workgroup: one slice of one row.
template <typename T, int kR, bool kEntropy, bool kTop>
__global__ __launch_bounds__(kVThreads) void k_vocab_slice(const T *__restrict__ Z, int V, int64_t ld, int S, int per,
                                                           float c, int top, Partial *__restrict__ part,
                                                           uint64_t *__restrict__ keys) {
  constexpr int n = Words<T>::n;
  __shared__ float sh[3][kVWaves];
  const int64_t m = blockIdx.x / S;
  const int sl = static_cast<int>(blockIdx.x % S);
  const Row<T> row(Z, ld, m, V);
  const int v0 = sl * per + static_cast<int>(threadIdx.x);
  const int v1 = sl * per + per;

  Vec<T> x[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int v = v0 + kVThreads * i;
    if (v < v1) {
      x[i] = row.load(v);
    } else {
#pragma unroll
      for (int e = 0; e < n; ++e) x[i].w[e] = static_cast<T>(-INFINITY);
    }
  }
  float top1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int e = 0; e < n; ++e) top1 = fmaxf(top1, as_f32(x[i].w[e]));
  const float zmax = block_max(top1, sh[0]);
  const float a = zmax == -INFINITY ? 0.f : zmax;
  float s = 0.f, u = 0.f;
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int e = 0; e < n; ++e) {
      const float t = (as_f32(x[i].w[e]) - a) * c;
      const float p = __builtin_amdgcn_exp2f(t);
      s += p;
      if (kEntropy) u = __builtin_fmaf(fmaxf(t, -300.f), p, u);
    }
  s = block_sum(s, sh[1]);
  if (kEntropy) u = block_sum(u, sh[2]);
  if (threadIdx.x == 0) part[m * S + sl] = Partial{zmax, s, u};

  if constexpr (kTop) {
    // The slice's `top` best.  A bound that at least `top` threads' maxima
    // reach is reached by every one of the `top` best words; bisection over
    // the ordered integers finds one that not many more reach.
    __shared__ uint32_t smax[kVThreads];
    __shared__ uint64_t cand[kCandMax];
    __shared__ int count;
    const uint32_t mine = ordered(top1);
    smax[threadIdx.x] = mine;
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    uint32_t g[kVThreads / 64];
#pragma unroll
    for (int w = 0; w < kVThreads / 64; ++w) g[w] = smax[64 * w + (threadIdx.x & 63)];
    auto reach = [&](uint32_t b) {
      int k = 0;
#pragma unroll
      for (int w = 0; w < kVThreads / 64; ++w) k += __popcll(__ballot(g[w] >= b));
      return k;
    };
    uint32_t lo = 0, hi = 0xFFFFFFFFu;   // reach(lo) >= top, reach(hi) < top
    int k = kVThreads;
    while (hi - lo > 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const int r = reach(mid);
      if (r >= top) {
        lo = mid;
        k = r;
        if (k <= top + top / 4) break;
      } else {
        hi = mid;
      }
    }
    const int j0 = row.first(sl * per) + static_cast<int>(threadIdx.x) * n;
    auto word = [&](int i, int e) { return j0 + i * kVThreads * n + e; };
    auto real = [&](int i, int j) { return j >= 0 && j < V && static_cast<int>(threadIdx.x) + kVThreads * i < per; };
    // Equal maxima in many threads (masked or flat rows): of the words that
    // equal the bound, only those up to the index jb that `top` threads reach.
    uint32_t jb = 0xFFFFFFFFu;
    if (k > top + top / 4) {
      uint32_t j1 = mine > lo ? 0u : 0xFFFFFFFFu;   // this thread's first word that equals the bound
#pragma unroll
      for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int e = 0; e < n; ++e) {
          const int j = word(i, e);
          if (mine == lo && ordered(as_f32(x[i].w[e])) == lo && real(i, j)) j1 = min(j1, static_cast<uint32_t>(j));
        }
      __syncthreads();
      smax[threadIdx.x] = ~j1;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kVThreads / 64; ++w) g[w] = smax[64 * w + (threadIdx.x & 63)];
      uint32_t a = 0, b = 0xFFFFFFFFu;
      if (reach(~(0xFFFFFFFFu - 1u)) >= top) {   // else fewer than `top` threads hold words: take all of them
        b = 0xFFFFFFFEu;
        while (a < b) {
          const uint32_t mid = a + (b - a) / 2;
          if (reach(~mid) >= top)
            b = mid;
          else
            a = mid + 1;
        }
      }
      jb = b;
    }
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const float z = as_f32(x[i].w[e]);
        const uint32_t o = ordered(z);
        if (o >= lo) {
          const int j = word(i, e);
          if (real(i, j) && (o > lo || static_cast<uint32_t>(j) <= jb)) {
            const int at = atomicAdd(&count, 1);
            if (at < kCandMax) cand[at] = word_key(z, static_cast<uint32_t>(j));
          }
        }
      }
    __syncthreads();
    uint64_t *out = keys + (m * S + sl) * top;
    const int found = count;
    if (found <= kCandMax) {
      // a candidate's place is the number of better ones (keys differ)
      for (int i = threadIdx.x; i < max(found, top); i += kVThreads) {
        if (i < found) {
          const uint64_t k = cand[i];
          int place = 0;
          for (int q = 0; q < found; ++q) place += cand[q] > k;
          if (place < top) out[place] = k;
        }
        if (i >= found && i < top) out[i] = 0;   // a slice shorter than `top`
      }
    } else {
      // Many words share the bound (a flat row): the next best one at a time.
      __shared__ uint64_t best[kVWaves];
      uint64_t last = ~uint64_t{0};
      for (int k = 0; k < top; ++k) {
        uint64_t b = 0;
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int e = 0; e < n; ++e) {
            const int j = word(i, e);
            if (real(i, j)) {
              const uint64_t key = word_key(as_f32(x[i].w[e]), static_cast<uint32_t>(j));
              if (key < last && key > b) b = key;
            }
          }
        for (int o = 32; o >= 1; o >>= 1) {
          const uint64_t other = __shfl_xor(b, o, 64);
          b = other > b ? other : b;
        }
        __syncthreads();
        if ((threadIdx.x & 63) == 0) best[threadIdx.x >> 6] = b;
        __syncthreads();
        for (int w = 0; w < kVWaves; ++w) b = best[w] > b ? best[w] : b;
        if (threadIdx.x == 0) out[k] = b;
        last = b;
      }
    }
  }
}

namespace {

// A row's sums from its slices', in 64 bits: the maximum, log s and the entropy.
struct RowSums {
  double a, logs, entropy;
  bool empty;   // all -inf
};

constexpr double kLn2 = 0.6931471805599453;

__device__ __forceinline__ RowSums join(const Partial *p, int S, float c) {
  float a = -INFINITY;
  for (int i = 0; i < S; ++i) a = fmaxf(a, p[i].a);
  RowSums o{a, 0.0, 0.0, a == -INFINITY};
  double s = 0.0, u = 0.0;
  for (int i = 0; i < S; ++i) {
    if (p[i].s == 0.f) continue;   // an all -inf slice: its a is no reference
    const double d = p[i].a == a ? 0.0 : (static_cast<double>(p[i].a) - static_cast<double>(a)) * static_cast<double>(c);
    const double f = exp2(d);
    s += f * p[i].s;
    u += f * (p[i].u + fmax(d, -1e6) * p[i].s);
  }
  if (o.empty) {
    o.logs = o.entropy = s;        // 0, or NaN where a NaN is the row's only number
  } else {
    const double l = log2(s);
    o.logs = l * kLn2;
    o.entropy = (l - u / s) * kLn2;
  }
  o.empty = o.empty && s == 0.0;
  return o;
}

// log p of a word.
__device__ __forceinline__ double log_p(const RowSums &o, float z, float temperature) {
  return o.empty ? -INFINITY : (static_cast<double>(z) - o.a) / static_cast<double>(temperature) - o.logs;
}

// The pair of a row.
__device__ __forceinline__ void put_lse(float *lse, int64_t m, const RowSums &o) {
  lse[2 * m] = static_cast<float>(o.a);
  lse[2 * m + 1] = static_cast<float>(o.logs);
}

}  // namespace

// One wave a row: its sums, the target's log probability, the entropy and the
// alternatives (each slice's list is sorted: a key's place is its place in
// its own list plus, in every other, the number of better keys).
template <typename T>
__global__ __launch_bounds__(64) void k_logprobs_join(const T *__restrict__ Z, int64_t V, int64_t ld, int S,
                                                      const int64_t *__restrict__ target, int top,
                                                      const Partial *__restrict__ part,
                                                      const uint64_t *__restrict__ keys, float *__restrict__ logprob,
                                                      float *__restrict__ entropy, float *__restrict__ lse,
                                                      float *__restrict__ top_logprob, int64_t *__restrict__ top_index) {
  const int64_t m = blockIdx.x;
  const RowSums o = join(part + m * S, S, kLog2e);
  if (threadIdx.x == 0) {
    const int64_t t = target[m];
    logprob[m] = (t >= 0 && t < V) ? static_cast<float>(log_p(o, as_f32(Z[m * ld + t]), 1.f)) : 0.f;
    entropy[m] = static_cast<float>(o.entropy);
    put_lse(lse, m, o);
  }
  const uint64_t *k = keys + m * S * top;
  for (int i = threadIdx.x; i < S * top; i += 64) {
    const uint64_t key = k[i];
    if (key == 0) continue;
    const int own = i / top;
    int place = i - own * top;
    for (int s = 0; s < S && place < top; ++s) {
      if (s == own) continue;
      int a = 0, b = top;   // keys before a are better, from b on they are not
      while (a < b) {
        const int mid = (a + b) / 2;
        if (k[s * top + mid] > key)
          a = mid + 1;
        else
          b = mid;
      }
      place += a;
    }
    if (place < top) {
      top_index[m * top + place] = key_index(key);
      top_logprob[m * top + place] = static_cast<float>(log_p(o, key_value(key), 1.f));
    }
  }
}

// Elementwise gradient kernels: a workgroup takes kGradVecs 16-byte vectors of
// one row.
constexpr int kGradVecs = 4 * kVThreads;

namespace {

// Stores the words of vector v that belong to the row.
template <typename T>
__device__ __forceinline__ void store_vec(T *row, int j, int V, const Vec<T> &x, bool same) {
  if (same && j >= 0 && j + Words<T>::n <= V) {
    *reinterpret_cast<Vec<T> *>(row + j) = x;
  } else {
#pragma unroll
    for (int e = 0; e < Words<T>::n; ++e)
      if (j + e >= 0 && j + e < V) row[j + e] = x.w[e];
  }
}

}  // namespace

template <typename T>
__global__ __launch_bounds__(kVThreads) void k_logprobs_bwd(const T *Z, int V, int64_t ld, int chunks,
                                                            const int64_t *__restrict__ target,
                                                            const float *__restrict__ lse,
                                                            const float *__restrict__ entropy,
                                                            const float *__restrict__ g_logprob,
                                                            const float *__restrict__ g_entropy, T *dZ, int64_t ldd) {
  constexpr int n = Words<T>::n;
  const int64_t m = blockIdx.x / chunks;
  const int v0 = static_cast<int>(blockIdx.x % chunks) * kGradVecs + static_cast<int>(threadIdx.x);
  const Row<T> row(Z, ld, m, V);
  T *out = dZ + m * ldd;
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(row.p) & 15);
  const int64_t t = target[m];
  const float a = lse[2 * m], logs = lse[2 * m + 1] * kLog2e;
  const bool empty = a == -INFINITY && logs == 0.f;
  const float gl = (t >= 0 && t < V && g_logprob && !empty) ? g_logprob[m] : 0.f;
  const float gh = g_entropy ? g_entropy[m] : 0.f;
  const float h = entropy[m];
  // with log p_j = q_j ln 2: dz_j = -p_j (g_lp + g_H (q_j ln 2 + H))
  const float g0 = gl + gh * h, g1 = gh * 0.693147182f;
  const float ref = a == -INFINITY ? 0.f : a;
#pragma unroll
  for (int i = 0; i < kGradVecs / kVThreads; ++i) {
    const int v = v0 + kVThreads * i;
    const int j = row.first(v);
    if (j >= V) break;
    const Vec<T> x = row.load(v);
    Vec<T> d;
#pragma unroll
    for (int e = 0; e < n; ++e) {
      const float q = __builtin_fmaf(as_f32(x.w[e]) - ref, kLog2e, -logs);
      const float p = __builtin_amdgcn_exp2f(q);
      float g = -p * __builtin_fmaf(g1, fmaxf(q, -300.f), g0);
      if (empty) g = 0.f;
      if (j + e == t) g += gl;
      d.w[e] = static_cast<T>(g);
    }
    store_vec(out, j, V, d, same);
  }
}

namespace {

// The teacher's side of a row: entry i's probability q_i (0 for no entry) and
// its logarithm, the entries of the row in threads' order.  Every thread of
// the workgroup takes part; K <= kDistillMax.
struct TeacherRow {
  float q[kDistillMax];       // q_i
  float total[kDistillMax];   // sum of the q of the entries with i's index, at its first one; 0 at the others
  int64_t idx[kDistillMax];   // -1 for no entry
  double loss[8];
  float any;
};

template <typename T>
__device__ __forceinline__ void teacher_row(TeacherRow &sh, const T *zrow, int64_t V, const Teacher &t, int64_t m,
                                              double &logq_out, float &z_out) {
  // wave 0 makes q: maximum, sum, quotient
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    float v[kDistillMax / 64];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kDistillMax / 64; ++i) {
      const int k = 64 * i + lane;
      v[i] = -INFINITY;
      if (k < t.K) {
        const int64_t j = t.idx[m * t.K + k];
        const bool real = j >= 0 && j < V;
        sh.idx[k] = real ? j : -1;
        if (real) v[i] = t.val[m * t.K + k];
      }
      top = fmaxf(top, v[i]);
    }
    top = wave_max(top);
    const double inv = 1.0 / static_cast<double>(t.temperature);
    double e[kDistillMax / 64], sum = 0.0;
#pragma unroll
    for (int i = 0; i < kDistillMax / 64; ++i) {
      e[i] = (top == -INFINITY || v[i] == -INFINITY)
                 ? 0.0
                 : exp((static_cast<double>(v[i]) - static_cast<double>(top)) * inv);
      sum += e[i];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
    const double lsum = sum > 0.0 ? log(sum) : 0.0;
#pragma unroll
    for (int i = 0; i < kDistillMax / 64; ++i) {
      const int k = 64 * i + lane;
      if (k < t.K) sh.q[k] = sum > 0.0 ? static_cast<float>(e[i] / sum) : (sum == 0.0 ? 0.f : NAN);
    }
    if (lane == 0) {
      sh.any = sum == 0.0 ? 0.f : 1.f;
      sh.loss[0] = static_cast<double>(top);
      sh.loss[1] = lsum;
    }
  }
  __syncthreads();
  const double top = sh.loss[0], lsum = sh.loss[1];
  const int k = threadIdx.x;
  logq_out = 0.0;
  z_out = 0.f;
  if (k < t.K) {
    const int64_t j = sh.idx[k];
    float total = 0.f;
    if (j >= 0) {
      logq_out = (static_cast<double>(t.val[m * t.K + k]) - top) / static_cast<double>(t.temperature) - lsum;
      z_out = as_f32(zrow[j]);
      bool first = true;
      for (int i = 0; i < t.K; ++i)
        if (sh.idx[i] == j) {
          first = first && i >= k;
          total += sh.q[i];
        }
      if (!first) total = 0.f;
    }
    sh.total[k] = total;
  }
  __syncthreads();
}

// Sum over the workgroup's first kDistillMax threads of q (log q - log p), in
// a fixed order; every thread gets it.
__device__ __forceinline__ double distill_loss(TeacherRow &sh, int K, double logq, double logp) {
  double v = 0.0;
  const int k = threadIdx.x;
  if (k < K && sh.idx[k] >= 0 && sh.q[k] != 0.f) v = static_cast<double>(sh.q[k]) * (logq - logp);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0 && threadIdx.x < kDistillMax) sh.loss[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kDistillMax / 64; ++w) s += sh.loss[w];
  return s;
}

}  // namespace

// One workgroup a row, after k_vocab_slice.
template <typename T>
__global__ __launch_bounds__(kDistillMax) void k_distill_join(const T *__restrict__ Z, int64_t V, int64_t ld, int S,
                                                              float c, Teacher t, const Partial *__restrict__ part,
                                                              float *__restrict__ loss, float *__restrict__ lse) {
  __shared__ TeacherRow sh;
  const int64_t m = blockIdx.x;
  const RowSums o = join(part + m * S, S, c);
  double logq;
  float z;
  teacher_row(sh, Z + m * ld, V, t, m, logq, z);
  const double v = distill_loss(sh, t.K, logq, log_p(o, z, t.temperature));
  if (threadIdx.x == 0) {
    loss[m] = sh.any == 0.f ? 0.f : static_cast<float>(v);
    put_lse(lse, m, o);
  }
}

namespace {

// The listed words' gradients, written over the row's after every wave's
// stores have been acknowledged: (p - total) scaled.
template <typename T>
__device__ __forceinline__ void patch_listed(const TeacherRow &sh, int K, float z, float c, float ref, float logs,
                                             float scale, int lo, int hi, T *out) {
  const int k = threadIdx.x;
  if (k < K && sh.total[k] != 0.f && scale != 0.f) {
    const int64_t j = sh.idx[k];
    if (j >= lo && j < hi) {
      const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(z - ref, c, -logs));
      out[j] = static_cast<T>((p - sh.total[k]) * scale);
    }
  }
}

__device__ __forceinline__ void stores_done() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

}  // namespace

template <typename T>
__global__ __launch_bounds__(kVThreads) void k_distill_bwd(const T *Z, int V, int64_t ld, int chunks, float c,
                                                           Teacher t, const float *__restrict__ lse,
                                                           const float *__restrict__ weight, T *dZ, int64_t ldd) {
  constexpr int n = Words<T>::n;
  __shared__ TeacherRow sh;
  const int64_t m = blockIdx.x / chunks;
  const int first = static_cast<int>(blockIdx.x % chunks) * kGradVecs;
  const Row<T> row(Z, ld, m, V);
  T *out = dZ + m * ldd;
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(row.p) & 15);
  double logq;
  float z;
  teacher_row(sh, row.p, V, t, m, logq, z);
  const float a = lse[2 * m], logs = lse[2 * m + 1] * kLog2e;
  const bool empty = a == -INFINITY && logs == 0.f;
  const float ref = a == -INFINITY ? 0.f : a;
  const float w = (weight ? weight[m] : 1.f) / t.temperature;
  const float scale = empty ? 0.f : w, pscale = sh.any == 0.f ? 0.f : scale;
#pragma unroll
  for (int i = 0; i < kGradVecs / kVThreads; ++i) {
    const int v = first + static_cast<int>(threadIdx.x) + kVThreads * i;
    const int j = row.first(v);
    if (j >= V) break;
    const Vec<T> x = row.load(v);
    Vec<T> d;
#pragma unroll
    for (int e = 0; e < n; ++e) {
      const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(as_f32(x.w[e]) - ref, c, -logs));
      d.w[e] = static_cast<T>(pscale == 0.f ? 0.f : p * pscale);
    }
    store_vec(out, j, V, d, same);
  }
  stores_done();
  patch_listed(sh, t.K, z, c, ref, logs, scale, max(row.first(first), 0),
               min(row.first(first + kGradVecs), V), out);
}

namespace {

template <typename T>
int grad_chunks(int64_t V) {
  const int64_t nv = (V + 2 * Words<T>::n - 2) / Words<T>::n;
  return static_cast<int>((nv + kGradVecs - 1) / kGradVecs);
}

template <typename T, bool kEntropy, bool kTop>
void launch_slice(const Logits &l, const Slices &sl, float c, int top, Partial *part, uint64_t *keys, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(l.M * sl.S));
  const T *z = static_cast<const T *>(l.z);
  const int vecs = (sl.per + kVThreads - 1) / kVThreads;
  constexpr int kFull = static_cast<int>(kSliceMax / Words<T>::n / kVThreads) + 1;
  if (vecs <= 2)
    hipLaunchKernelGGL((k_vocab_slice<T, 2, kEntropy, kTop>), grid, dim3(kVThreads), 0, s, z, static_cast<int>(l.V), l.ld, sl.S, sl.per,
                       c, top, part, keys);
  else
    hipLaunchKernelGGL((k_vocab_slice<T, kFull, kEntropy, kTop>), grid, dim3(kVThreads), 0, s, z, static_cast<int>(l.V), l.ld, sl.S,
                       sl.per, c, top, part, keys);
}

template <typename T>
hipError_t logprobs_as(const Logits &l, const int64_t *target, int top, float *logprob, float *entropy, float *lse,
                       float *top_logprob, int64_t *top_index, void *ws, hipStream_t s) {
  const Slices sl = slices_of(l.M, l.V, l.type);
  Partial *part = static_cast<Partial *>(ws);
  uint64_t *keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) +
                                                up256(static_cast<size_t>(l.M) * sl.S * sizeof(Partial)));
  if (top)
    launch_slice<T, true, true>(l, sl, kLog2e, top, part, keys, s);
  else
    launch_slice<T, true, false>(l, sl, kLog2e, top, part, keys, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_logprobs_join<T>, dim3(static_cast<uint32_t>(l.M)), dim3(64), 0, s, static_cast<const T *>(l.z),
                     l.V, l.ld, sl.S, target, top, part, keys, logprob, entropy, lse, top_logprob, top_index);
  return hipGetLastError();
}

template <typename T>
hipError_t logprobs_bwd_as(const Logits &l, const int64_t *target, const float *lse, const float *entropy,
                           const float *g_logprob, const float *g_entropy, void *dz, int64_t ldd, hipStream_t s) {
  const int chunks = grad_chunks<T>(l.V);
  hipLaunchKernelGGL(k_logprobs_bwd<T>, dim3(static_cast<uint32_t>(l.M * chunks)), dim3(kVThreads), 0, s,
                     static_cast<const T *>(l.z), static_cast<int>(l.V), l.ld, chunks, target, lse, entropy, g_logprob, g_entropy,
                     static_cast<T *>(dz), ldd);
  return hipGetLastError();
}

float scaled_log2e(float temperature) {
  return static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
}

template <typename T>
hipError_t distill_fwd_as(const Logits &l, const Teacher &t, float *loss, float *lse, void *ws, hipStream_t s) {
  const Slices sl = slices_of(l.M, l.V, l.type);
  const float c = scaled_log2e(t.temperature);
  Partial *part = static_cast<Partial *>(ws);
  launch_slice<T, false, false>(l, sl, c, 0, part, nullptr, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_distill_join<T>, dim3(static_cast<uint32_t>(l.M)), dim3(kDistillMax), 0, s,
                     static_cast<const T *>(l.z), l.V, l.ld, sl.S, c, t, part, loss, lse);
  return hipGetLastError();
}

template <typename T>
hipError_t distill_bwd_as(const Logits &l, const Teacher &t, const float *lse, const float *weight, void *dz,
                          int64_t ldd, hipStream_t s) {
  const int chunks = grad_chunks<T>(l.V);
  hipLaunchKernelGGL(k_distill_bwd<T>, dim3(static_cast<uint32_t>(l.M * chunks)), dim3(kVThreads), 0, s,
                     static_cast<const T *>(l.z), static_cast<int>(l.V), l.ld, chunks, scaled_log2e(t.temperature), t, lse, weight,
                     static_cast<T *>(dz), ldd);
  return hipGetLastError();
}

}  // namespace

#define QLORA_BY_TYPE(type, call)              \
  switch (type) {                              \
    case 0: { using T = float; return call; }  \
    case 1: { using T = __bf16; return call; } \
    default: { using T = _Float16; return call; } \
  }

hipError_t launch_token_logprobs(const Logits &l, const int64_t *target, int top, float *logprob, float *entropy,
                                 float *lse, float *top_logprob, int64_t *top_index, void *ws, hipStream_t s) {
  QLORA_BY_TYPE(l.type, logprobs_as<T>(l, target, top, logprob, entropy, lse, top_logprob, top_index, ws, s))
}

hipError_t launch_token_logprobs_bwd(const Logits &l, const int64_t *target, const float *lse, const float *entropy,
                                     const float *g_logprob, const float *g_entropy, void *dz, int64_t ldd,
                                     hipStream_t s) {
  QLORA_BY_TYPE(l.type, logprobs_bwd_as<T>(l, target, lse, entropy, g_logprob, g_entropy, dz, ldd, s))
}

hipError_t launch_distill_fwd(const Logits &l, const Teacher &t, float *loss, float *lse, void *ws, hipStream_t s) {
  QLORA_BY_TYPE(l.type, distill_fwd_as<T>(l, t, loss, lse, ws, s))
}

hipError_t launch_distill_bwd(const Logits &l, const Teacher &t, const float *lse, const float *weight, void *dz,
                              int64_t ldd, hipStream_t s) {
  QLORA_BY_TYPE(l.type, distill_bwd_as<T>(l, t, lse, weight, dz, ldd, s))
}

hipError_t launch_distill(const Logits &l, const Teacher &t, const float *weight, float *loss, float *lse, void *dz,
                          int64_t ldd, void *ws, hipStream_t s) {
  const hipError_t e = launch_distill_fwd(l, t, loss, lse, ws, s);
  return e != hipSuccess ? e : launch_distill_bwd(l, t, lse, weight, dz, ldd, s);
}

#undef QLORA_BY_TYPE

}  // namespace qlora
