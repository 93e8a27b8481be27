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
// A workgroup holds its words in registers, 8 16-byte vectors a thread, so that
// z is read once for the maximum, the sums and the alternatives, and by the
// fused distillation for the gradient too.  A row that fits one workgroup of
// up to 1024 threads (65536 16-bit words) is finished there, in one launch; a
// longer row, or one of few long ones, is cut into slices that a second kernel
// joins.  The order of every sum is fixed.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr int kVThreads = 256;          // of a slice and of the gradient kernels
constexpr int kVecs = 8;                // 16-byte vectors a thread holds
constexpr int kGroups = 256;            // threads' maxima are grouped into these for the alternatives
constexpr int kCandMax = 1024;          // alternatives considered by a workgroup
constexpr int kJoinMax = 2048;          // and by the join of a row
constexpr float kLog2e = 1.44269502f;   // fp32 nearest to log2(e)
constexpr double kLn2 = 0.6931471805599453;

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__bf16 v) { return static_cast<float>(v); }
__device__ __forceinline__ float as_f32(_Float16 v) { return static_cast<float>(v); }

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// A 16-byte vector of words, kept as four registers: arrays of 16-bit types
// would take one a word.
template <typename T>
struct Words {
  static constexpr int n = 16 / static_cast<int>(sizeof(T));
  static constexpr uint32_t kMasked = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __bf16>::value ? 0xFF80FF80u : 0xFC00FC00u;
  uint32_t r[4];

  __device__ __forceinline__ float get(int e) const {
    if (sizeof(T) == 4) return __uint_as_float(r[e]);
    if (std::is_same<T, __bf16>::value) return __uint_as_float((e & 1) ? r[e >> 1] & 0xFFFF0000u : r[e >> 1] << 16);
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(r[e >> 1] >> (16 * (e & 1)))));
  }
  __device__ __forceinline__ T raw(int e) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(r[e]);
    else
      return __builtin_bit_cast(T, static_cast<uint16_t>(r[e >> 1] >> (16 * (e & 1))));
  }
  // From fp32, words 2 i and 2 i + 1 (16-bit types), rounded to nearest even.
  __device__ __forceinline__ void put(const float (&v)[n]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        r[i] = __float_as_uint(v[i]);
      } else {
        typedef T pair __attribute__((ext_vector_type(2)));
        const pair w = {static_cast<T>(v[2 * i]), static_cast<T>(v[2 * i + 1])};
        r[i] = __builtin_bit_cast(uint32_t, w);
      }
    }
  }
  __device__ __forceinline__ void mask() {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = kMasked;
  }
};

// Row m of a matrix cut at 16-byte boundaries: vector v covers words v n -
// mis .. of the row, mis = the row's first word within its 16 bytes.
// Vectors whole .. ends - 1 lie inside the row; one before and one after
// them may be cut by its ends.
template <typename T>
struct Row {
  static constexpr int n = Words<T>::n;
  const T *p;
  int V, mis, whole, ends;
  __device__ __forceinline__ Row(const T *base, int64_t ld, int64_t m, int v) : p(base + m * ld), V(v) {
    mis = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    whole = mis > 0;
    ends = (V + mis) / n;
  }
  __device__ __forceinline__ int first(int v) const { return v * n - mis; }
  __device__ __forceinline__ bool inside(int v) const { return v >= whole && v < ends; }
  __device__ __forceinline__ const u32x4_t *at(int v) const {
    const char *b = reinterpret_cast<const char *>(p - mis);   // uniform; the lane's part is a 32-bit offset
    return reinterpret_cast<const u32x4_t *>(b + static_cast<uint32_t>(v) * 16u);
  }
  __device__ __forceinline__ Words<T> load_inside(int v) const {
    const u32x4_t w = *at(v);
    return Words<T>{{w[0], w[1], w[2], w[3]}};
  }
  // Read once and not kept in the L2: 157 us instead of 212 for the sums of
  // 4096 rows of 131072 bf16 words (6.8 TB/s), 44 instead of 72 for 1024.
  __device__ __forceinline__ Words<T> load_once(int v) const {
    const u32x4_t w = __builtin_nontemporal_load(at(v));
    return Words<T>{{w[0], w[1], w[2], w[3]}};
  }
  // Words outside the row are -inf; only words of the row are read.
  __device__ __forceinline__ Words<T> load_cut(int v) const {
    const int j = first(v);
    float w[n];
#pragma unroll
    for (int e = 0; e < n; ++e) w[e] = (j + e >= 0 && j + e < V) ? as_f32(p[j + e]) : -INFINITY;
    Words<T> x;
    x.put(w);   // exact: the values are of type T
    return x;
  }
  __device__ __forceinline__ Words<T> load(int v) const { return inside(v) ? load_inside(v) : load_cut(v); }
};

// max(a, b, c) in one instruction: fmaxf on unpacked words would first quiet
// each of them.  A NaN is passed over or kept; its row's sums are NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

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
// Order-preserving integer of a float (-0 as +0).  A NaN counts as -inf, as in
// the maxima, which pass over it: every word can be an alternative, and a row
// always has enough of them.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v == v ? v + 0.f : -INFINITY);
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

// The words of a workgroup: vectors v0 + threadIdx.x + NT i of a row.
template <typename T, int NT>
struct Held {
  Words<T> x[kVecs];

  // Whether vectors v0 + NT i .. + NT - 1 all lie in the workgroup's part and
  // inside the row: then nothing is tested a lane.
  static __device__ __forceinline__ bool full(const Row<T> &row, int v0, int per, int i) {
    return NT * (i + 1) <= per && v0 + NT * i >= row.whole && v0 + NT * (i + 1) <= row.ends;
  }
  // All loads first, in one straight line (a branch around each would wait for
  // it): a lane without a vector reads the row's nearest whole one, and is
  // masked afterwards.
  __device__ __forceinline__ void load(const Row<T> &row, int v0, int per) {
    const int tid = static_cast<int>(threadIdx.x);
    if (row.ends > row.whole) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) x[i] = row.load_once(min(max(v0 + tid + NT * i, row.whole), row.ends - 1));
    }
    // the row's cut vectors: the first (the row's first workgroup, thread 0) and the last
    const int last = row.ends - v0;
    const bool has_head = row.whole && v0 == 0 && tid == 0;
    const bool has_tail = last >= 0 && last < per && (row.V + row.mis) % Words<T>::n != 0 && tid == last % NT;
    Words<T> head, tail;
    head.mask();
    tail.mask();
    if (has_head) head = row.load_cut(0);
    if (has_tail) tail = row.load_cut(row.ends);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (full(row, v0, per, i)) continue;
      const bool ok = tid + NT * i < per && row.inside(v0 + tid + NT * i);
      const bool is_tail = has_tail && i == last / NT;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w = ok ? x[i].r[q] : Words<T>::kMasked;
        if (i == 0) w = has_head ? head.r[q] : w;
        x[i].r[q] = is_tail ? tail.r[q] : w;
      }
    }
  }
  // Forget what the compiler knows of the words: unpacked copies are not kept
  // from one pass over them to the next (they would double the registers).
  __device__ __forceinline__ void again() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      asm volatile("" : "+v"(x[i].r[0]), "+v"(x[i].r[1]), "+v"(x[i].r[2]), "+v"(x[i].r[3]));
    }
  }
  // The maximum, and of each vector.
  __device__ __forceinline__ float maximum(float (&vm)[kVecs], int per) const {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      vm[i] = -INFINITY;
      if (NT * i >= per) continue;
#pragma unroll
      for (int e = 0; e < Words<T>::n; e += 2) vm[i] = max3(vm[i], x[i].get(e), x[i].get(e + 1));
      m = fmaxf(m, vm[i]);
    }
    return m;
  }
  // Zeros for the words.
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[i].r[q] = 0;
  }
  // Vector i of the thread, i known at run time only.
  __device__ __forceinline__ Words<T> pick(int i) const {
    Words<T> w = x[0];
#pragma unroll
    for (int k = 1; k < kVecs; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) w.r[q] = i == k ? x[k].r[q] : w.r[q];
    return w;
  }
};

// 2^t of the words, t = (z - a) c.  One fused multiply-add by r = fl(a c);
// dr = a c - r is what that rounding changed, the same for every word, and the
// sums are relative to 2^dr (see corrected).  Up to |r| = kNear |dr| is 2^-9 at
// most, so nothing leaves fp32's range and the correction costs no digits.
// Beyond (masks by a finite value of any size, small temperatures) the
// difference comes first, which is as exact and one operation more; the choice
// is the same for a whole workgroup.
constexpr float kNear = 65536.f;
struct Exps {
  float a, c, r, dr;
  bool far;
  __device__ __forceinline__ Exps(float zmax, float scale) : a(zmax == -INFINITY ? 0.f : zmax), c(scale) {
    r = a * c;
    far = !(fabsf(r) < kNear);
    dr = far ? 0.f : __builtin_fmaf(a, c, -r);
  }
  template <bool kFar>
  __device__ __forceinline__ float t(float z) const {
    return kFar ? (z - a) * c : __builtin_fmaf(z, c, -r);
  }
};

// kMasked: -inf among the words (0 * -inf in u); needed only where the plain
// sum came out as a NaN, so a wave without masked words never pays for it.
template <bool kFar, bool kEntropy, bool kMasked, typename T, int NT>
__device__ __forceinline__ void thread_sums(const Held<T, NT> &h, const Exps &x, int per, float &s, float &u) {
  s = u = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (NT * i >= per) continue;
#pragma unroll
    for (int e = 0; e < Words<T>::n; ++e) {
      const float t = x.t<kFar>(h.x[i].get(e));
      const float p = __builtin_amdgcn_exp2f(t);
      s += p;
      if (kEntropy) u = __builtin_fmaf(kMasked ? fmaxf(t, -300.f) : t, p, u);
    }
  }
}

// Sums over the workgroup, every thread gets them; sh: two floats a wave.
template <bool kEntropy, int NT, typename T>
__device__ __forceinline__ void block_sums(Held<T, NT> &h, const Exps &x, int per, float &s, float &u, float (*sh)[2]) {
  h.again();
  if (x.far) {
    thread_sums<true, kEntropy, true>(h, x, per, s, u);
  } else {
    thread_sums<false, kEntropy, false>(h, x, per, s, u);
    if (kEntropy && __any(u != u)) thread_sums<false, true, true>(h, x, per, s, u);
  }
  s = wave_sum(s);
  if (kEntropy) u = wave_sum(u);
  if ((threadIdx.x & 63) == 0) {
    sh[threadIdx.x >> 6][0] = s;
    sh[threadIdx.x >> 6][1] = u;
  }
  __syncthreads();
  s = sh[0][0];
  u = sh[0][1];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) {
    s += sh[w][0];
    if (kEntropy) u += sh[w][1];
  }
}

// The `top` best of a workgroup's words, as falling keys to out (0: the
// workgroup has fewer words).  The threads' maxima are grouped; a bound that
// at least `top` groups reach is reached by every one of the `top` best
// words, and bisection over the ordered integers finds one that not many more
// reach: the words above it are few.  zmax: the workgroup's maximum, mine: the
// thread's.
struct TopShared {
  uint32_t smax[kGroups];
  uint64_t cand[kCandMax];
  uint64_t best[16];
  int count;
};

template <typename T, int NT>
__device__ __forceinline__ void block_top(Held<T, NT> &h, const float (&vm)[kVecs], const Row<T> &row, int v0, int per,
                                          float zmax, float thread_max, int top, TopShared &sh, uint64_t *out) {
  constexpr int n = Words<T>::n;
  constexpr int kPer = NT / kGroups;   // threads of a group
  const int tid = static_cast<int>(threadIdx.x);
  const uint32_t own = ordered(thread_max);
  uint32_t mine = own;
#pragma unroll
  for (int o = 1; o < kPer; o *= 2) mine = max(mine, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mine), o, 64)));
  if (tid % kPer == 0) sh.smax[tid / kPer] = mine;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  uint32_t g[kGroups / 64];
  auto gather = [&]() {
#pragma unroll
    for (int w = 0; w < kGroups / 64; ++w) g[w] = sh.smax[64 * w + (tid & 63)];
  };
  auto reach = [&](uint32_t b) {
    int k = 0;
#pragma unroll
    for (int w = 0; w < kGroups / 64; ++w) k += __popcll(__ballot(g[w] >= b));
    return k;
  };
  // f(word, index) for the thread's words in vectors whose maximum reaches b.
  auto words = [&](float b, auto f) __attribute__((always_inline)) {
    uint32_t todo = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) todo |= (tid + NT * i < per && !(vm[i] < b)) ? 1u << i : 0u;
    while (todo) {
      const int i = __builtin_ctz(todo);
      todo &= todo - 1;
      const Words<T> x = h.pick(i);
      const int j = row.first(v0 + tid + NT * i);
#pragma unroll
      for (int e = 0; e < n; ++e)
        if (j + e >= 0 && j + e < row.V) f(x.get(e), static_cast<uint32_t>(j + e));
    }
  };
  gather();
  uint32_t lo = 0, hi = ordered(zmax) + 1;   // reach(lo) >= top, reach(hi) < top
  int k = kGroups;
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
  const float bound = __uint_as_float((lo & 0x80000000u) ? (lo & 0x7FFFFFFFu) : ~lo);
  // Equal maxima in many groups (masked or flat rows): of the words that equal
  // the bound, only those up to the index jb that `top` groups reach.
  uint32_t jb = 0xFFFFFFFFu;
  if (k > top + top / 4) {
    uint32_t j1 = own > lo ? 0u : 0xFFFFFFFFu;   // this thread's first word that equals the bound
    if (own == lo) words(bound, [&](float z, uint32_t j) { j1 = ordered(z) == lo ? min(j1, j) : j1; });
#pragma unroll
    for (int o = 1; o < kPer; o *= 2) j1 = min(j1, static_cast<uint32_t>(__shfl_xor(static_cast<int>(j1), o, 64)));
    __syncthreads();
    if (tid % kPer == 0) sh.smax[tid / kPer] = ~j1;
    __syncthreads();
    gather();
    if (reach(~0xFFFFFFFEu) >= top) {   // else fewer than `top` groups hold words: take all of them
      uint32_t a = 0, b = 0xFFFFFFFEu;
      while (a < b) {
        const uint32_t mid = a + (b - a) / 2;
        if (reach(~mid) >= top)
          b = mid;
        else
          a = mid + 1;
      }
      jb = b;
    }
  }
  if (own >= lo)
    words(bound, [&](float z, uint32_t j) {
      const uint32_t o = ordered(z);
      if (o > lo || (o == lo && j <= jb)) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < kCandMax) sh.cand[at] = word_key(z, j);
      }
    });
  __syncthreads();
  const int found = sh.count;
  if (found <= kCandMax) {
    // a candidate's place is the number of better ones (keys differ)
    for (int i = tid; i < max(found, top); i += NT) {
      if (i < found) {
        const uint64_t key = sh.cand[i];
        int place = 0;
        for (int q = 0; q < found; ++q) place += sh.cand[q] > key;
        if (place < top) out[place] = key;
      } else {
        out[i] = 0;
      }
    }
  } else {
    // More than kCandMax words above the bound (rows whose best words lie in
    // few threads): the next best one at a time.
    uint64_t last = ~uint64_t{0};
    for (int q = 0; q < top; ++q) {
      uint64_t b = 0;
      if (own >= lo)
        words(bound, [&](float z, uint32_t j) {
          const uint64_t key = word_key(z, j);
          b = key < last && key > b ? key : b;
        });
      for (int o = 32; o >= 1; o >>= 1) {
        const uint64_t other = __shfl_xor(b, o, 64);
        b = other > b ? other : b;
      }
      __syncthreads();
      if ((tid & 63) == 0) sh.best[tid >> 6] = b;
      __syncthreads();
      for (int w = 0; w < NT / 64; ++w) b = sh.best[w] > b ? sh.best[w] : b;
      if (tid == 0) out[q] = b;
      last = b;
    }
  }
}

// A row's sums, in 64 bits: the maximum, log s and the entropy.
struct RowSums {
  double a, logs, entropy;
  bool empty;   // all -inf
};

__device__ __forceinline__ RowSums row_sums(float a, double s, double u) {
  RowSums o{a, s, s, false};      // 0, or NaN where a NaN is the row's only number
  if (a == -INFINITY) {
    o.empty = s == 0.0;
  } else {
    const double l = log2(s);
    o.logs = l * kLn2;
    o.entropy = (l - u / s) * kLn2;
  }
  return o;
}

// One workgroup's sums, relative to a itself (see Exps).
__device__ __forceinline__ Partial corrected(const Exps &x, float zmax, float s, float u) {
  const float f = __builtin_amdgcn_exp2f(-x.dr);
  return Partial{zmax, s * f, (u - x.dr * s) * f};
}

// Slices joined by a wave, lane by lane and then over the lanes.
__device__ __forceinline__ RowSums join(const Partial *p, int S, float c) {
  const int lane = threadIdx.x & 63;
  float a = -INFINITY;
  for (int i = lane; i < S; i += 64) a = fmaxf(a, p[i].a);
  a = wave_max(a);
  double s = 0.0, u = 0.0;
  for (int i = lane; i < S; i += 64) {
    const Partial q = p[i];
    if (q.s == 0.f) continue;   // an all -inf slice: its a is no reference
    const double d = q.a == a ? 0.0 : (static_cast<double>(q.a) - static_cast<double>(a)) * static_cast<double>(c);
    const double f = d == 0.0 ? 1.0 : exp2(d);
    s += f * q.s;
    u += f * (q.u + fmax(d, -1e6) * q.s);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    s += __shfl_xor(s, o, 64);
    u += __shfl_xor(u, o, 64);
  }
  return row_sums(a, s, u);
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

struct LogprobOut {
  float *logprob, *entropy, *lse, *top_logprob;
  int64_t *top_index;
};

template <typename T>
__device__ __forceinline__ void put_logprobs(const LogprobOut &out, const T *zrow, int V, int64_t m, int64_t t,
                                             const RowSums &o) {
  out.logprob[m] = (t >= 0 && t < V) ? static_cast<float>(log_p(o, as_f32(zrow[t]), 1.f)) : 0.f;
  out.entropy[m] = static_cast<float>(o.entropy);
  put_lse(out.lse, m, o);
}

__device__ __forceinline__ void put_top(const LogprobOut &out, int64_t at, uint64_t key, const RowSums &o) {
  out.top_index[at] = key_index(key);
  out.top_logprob[at] = static_cast<float>(log_p(o, key_value(key), 1.f));
}

// Slices of a launch and the workspace they leave: partials [M][S], then the
// alternatives' keys [M][S][top].
struct Slices {
  int S;             // slices of a row; 1: the row is finished by one workgroup
  int per;           // 16-byte vectors of a slice
  int threads;
};

// One workgroup a row where it fits: of 512 threads (one row of 32000 words in
// bf16, 5 alternatives: 9.6 us, as slices and a join 13.3; 128 rows: 13.1 and
// 20.3), or of 1024 (128 rows of 50000: logprobs 22.1 and 23.5, distill 16.9 and
// 24.8; 2048 rows: distill 133 and 147).  But 1024 threads are a workgroup a
// CU, with nothing to run beside its search for alternatives, so with those
// and more than a row a CU the row is cut (512 rows of 50000: 33.6 us, whole
// 40.5; 2048 rows: 88, whole 136).
Slices slices_of(int64_t M, int64_t V, int type, int top, bool aligned) {
  const int n = type == 0 ? 4 : 8;
  // a row that starts inside 16 bytes may touch one vector more
  const int nv = static_cast<int>((V + n - 1 + (aligned ? 0 : n - 1)) / n);
  constexpr int kSlice = kVThreads * kVecs;
  if (nv <= 2 * kSlice || (nv <= 4 * kSlice && (top == 0 || M <= 256)))
    return Slices{1, nv, nv <= kSlice ? 256 : nv <= 2 * kSlice ? 512 : 1024};
  // slices enough for two workgroups a CU, of one vector a thread at least,
  // and whole vectors for every thread
  const int64_t least = (nv + kSlice - 1) / kSlice, most = (nv + kVThreads - 1) / kVThreads;
  const int64_t want = std::max(least, std::min(most, (512 + M - 1) / std::max<int64_t>(M, 1)));
  const int per = static_cast<int>(((nv + want - 1) / want + kVThreads - 1) / kVThreads * kVThreads);
  return Slices{(nv + per - 1) / per, per, kVThreads};
}

Slices slices_of(const Logits &l, int top) {
  const bool aligned = (reinterpret_cast<uintptr_t>(l.z) & 15) == 0 && (l.M == 1 || l.ld % (l.type == 0 ? 4 : 8) == 0);
  return slices_of(l.M, l.V, l.type, top, aligned);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

size_t slices_bytes(int64_t M, const Slices &sl, int top) {
  if (sl.S == 1) return 0;
  return up256(static_cast<size_t>(M) * sl.S * sizeof(Partial)) + static_cast<size_t>(M) * sl.S * top * sizeof(uint64_t);
}

}  // namespace

size_t vocab_ws_bytes(int64_t M, int64_t V, int type, int top) {   // wherever the rows start
  return std::max(slices_bytes(M, slices_of(M, V, type, top, true), top), slices_bytes(M, slices_of(M, V, type, top, false), top));
}

// One workgroup: one slice of one row.  Bound by its one read: 4096 rows of
// 131072 bf16 words 158 to 167 us, 6.4 to 6.8 TB/s.
template <typename T, bool kEntropy, bool kTop>
__global__ __launch_bounds__(kVThreads, kTop ? 6 : 8) void k_vocab_slice(const T *__restrict__ Z, int V, int64_t ld, int S, int per,
                                                           float c, int top, Partial *__restrict__ part,
                                                           uint64_t *__restrict__ keys) {
  __shared__ float sh_max[kVThreads / 64], sh_sum[kVThreads / 64][2];
  const int64_t m = blockIdx.x / S;
  const int sl = static_cast<int>(blockIdx.x % S);
  const Row<T> row(Z, ld, m, V);
  Held<T, kVThreads> h;
  h.load(row, sl * per, per);
  float vm[kVecs];
  const float mine = h.maximum(vm, per);
  const float zmax = block_max(mine, sh_max);
  const Exps x(zmax, c);
  float s, u;
  block_sums<kEntropy>(h, x, per, s, u, sh_sum);
  if (threadIdx.x == 0) part[m * S + sl] = corrected(x, zmax, s, u);
  if constexpr (kTop) {
    __shared__ TopShared sh;
    block_top(h, vm, row, sl * per, per, zmax, mine, top, sh, keys + (m * S + sl) * top);
  }
}

// One workgroup: one row, finished.  4096 rows of 32000 bf16 words 50 us (5.2
// TB/s; with 64 alternatives 8192 rows 177); one row with 20 of them 10.5 us, a
// chain of one load, three block reductions and the search.
template <typename T, int NT, bool kTop>
__global__ __launch_bounds__(NT, kTop ? (NT == 1024 ? 4 : 6) : 8) void k_logprobs_row(const T *__restrict__ Z, int V, int64_t ld, int per,
                                                     const int64_t *__restrict__ target, int top, LogprobOut out) {
  __shared__ float sh_max[NT / 64], sh_sum[NT / 64][2];
  const int64_t m = blockIdx.x;
  const Row<T> row(Z, ld, m, V);
  Held<T, NT> h;
  h.load(row, 0, per);
  const int64_t t = target[m];
  float vm[kVecs];
  const float mine = h.maximum(vm, per);
  const float zmax = block_max(mine, sh_max);
  const Exps x(zmax, kLog2e);
  float s, u;
  block_sums<true>(h, x, per, s, u, sh_sum);
  if constexpr (kTop) {
    __shared__ TopShared sh;
    __shared__ uint64_t keys[kTopMax];
    block_top(h, vm, row, 0, per, zmax, mine, top, sh, keys);
    __syncthreads();
    if (threadIdx.x < 64) {
      const Partial p = corrected(x, zmax, s, u);
      const RowSums o = row_sums(p.a, p.s, p.u);
      if (threadIdx.x == 0) put_logprobs(out, row.p, V, m, t, o);
      if (static_cast<int>(threadIdx.x) < top) put_top(out, m * top + threadIdx.x, keys[threadIdx.x], o);
    }
  } else if (threadIdx.x == 0) {
    const Partial p = corrected(x, zmax, s, u);
    put_logprobs(out, row.p, V, m, t, row_sums(p.a, p.s, p.u));
  }
}

// A row's slices joined: one wave without alternatives, kVThreads threads with.
template <typename T, bool kTop>
__global__ __launch_bounds__(kTop ? kVThreads : 64) void k_logprobs_join(const T *__restrict__ Z, int V, int64_t ld, int S,
                                                                         const int64_t *__restrict__ target, int top,
                                                                         const Partial *__restrict__ part,
                                                                         const uint64_t *__restrict__ keys,
                                                                         LogprobOut out) {
  const int64_t m = blockIdx.x;
  const RowSums o = join(part + m * S, S, kLog2e);
  if (threadIdx.x == 0) put_logprobs(out, Z + m * ld, V, m, target[m], o);
  if constexpr (kTop) {
    __shared__ uint64_t cand[kJoinMax];
    __shared__ uint64_t smax[kVThreads];
    __shared__ int count;
    const uint64_t *k = keys + m * S * top;
    const int tid = static_cast<int>(threadIdx.x);
    // As in block_top, on whole keys: a bound that `top` threads' best keys
    // reach and not many more.  Entry q of list s goes to thread s + q odd: the
    // lists' first entries to different threads, and so those of one list.
    const int odd = S | 1, places = odd * top;
    auto entry = [&](int i) { return i % odd < S ? k[i % odd * top + i / odd] : uint64_t{0}; };
    uint64_t mine = 0;
    for (int i = tid; i < places; i += kVThreads) mine = max(mine, entry(i));
    smax[tid] = mine;
    if (tid == 0) count = 0;
    __syncthreads();
    uint64_t g[kVThreads / 64];
#pragma unroll
    for (int w = 0; w < kVThreads / 64; ++w) g[w] = smax[64 * w + (tid & 63)];
    uint64_t lo = 0, hi = ~uint64_t{0};   // as many as `top` reach lo, fewer reach hi
    while (hi - lo > 1) {
      const uint64_t mid = lo + (hi - lo) / 2;
      int r = 0;
#pragma unroll
      for (int w = 0; w < kVThreads / 64; ++w) r += __popcll(__ballot(g[w] >= mid));
      if (r >= top) {
        lo = mid;
        if (r <= top + top / 4) break;
      } else {
        hi = mid;
      }
    }
    const uint64_t bound = max(lo, uint64_t{1});   // 0 is no key
    if (mine >= bound)
      for (int i = tid; i < places; i += kVThreads) {
        const uint64_t key = entry(i);
        if (key >= bound) {
          const int at = atomicAdd(&count, 1);
          if (at < kJoinMax) cand[at] = key;
        }
      }
    __syncthreads();
    const int found = count;
    if (found <= kJoinMax) {
      for (int i = threadIdx.x; i < found; i += kVThreads) {
        const uint64_t key = cand[i];
        int place = 0;
        for (int q = 0; q < found; ++q) place += cand[q] > key;
        if (place < top) put_top(out, m * top + place, key, o);
      }
    } else {
      // More keys above the bound (rows whose best words lie in few slices): a
      // key's place is its place in its own list and, in every other, the number
      // of better keys there.
      for (int i = threadIdx.x; i < S * top; i += kVThreads) {
        const uint64_t key = k[i];
        if (key < bound) continue;
        const int own = i / top;
        int place = i - own * top;
        for (int s = 0; s < S && place < top; ++s) {
          if (s == own) continue;
          int lo = 0, hi = top;   // keys before lo are better, from hi on they are not
          while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (k[s * top + mid] > key)
              lo = mid + 1;
            else
              hi = mid;
          }
          place += lo;
        }
        if (place < top) put_top(out, m * top + place, key, o);
      }
    }
  }
}

// Elementwise gradient kernels: a workgroup takes kGradVecs 16-byte vectors of
// one row.
constexpr int kGradVecs = 4 * kVThreads;

namespace {

// Stores vector v of a row, inside it and 16-byte aligned as the one it came from.
template <typename T>
__device__ __forceinline__ void store_inside(T *row, int mis, int v, const float (&d)[Words<T>::n]) {
  Words<T> x;
  x.put(d);
  char *b = reinterpret_cast<char *>(row - mis);
  *reinterpret_cast<uint4 *>(b + static_cast<uint32_t>(v) * 16u) = make_uint4(x.r[0], x.r[1], x.r[2], x.r[3]);
}

// Stores the words of vector v that belong to the row.
template <typename T>
__device__ __forceinline__ void store_vec(T *row, int j, int V, const float (&d)[Words<T>::n], bool same) {
  Words<T> x;
  x.put(d);
  if (same && j >= 0 && j + Words<T>::n <= V) {
    *reinterpret_cast<uint4 *>(row + j) = make_uint4(x.r[0], x.r[1], x.r[2], x.r[3]);
  } else {
#pragma unroll
    for (int e = 0; e < Words<T>::n; ++e)
      if (j + e >= 0 && j + e < V) row[j + e] = x.raw(e);
  }
}

}  // namespace

// Read and written once: 4096 rows of 131072 bf16 words 360 to 379 us (5.7 to 6.0
// TB/s).
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
    const Words<T> x = row.load(v);
    float d[n];
#pragma unroll
    for (int e = 0; e < n; ++e) {
      const float q = __builtin_fmaf(x.get(e) - ref, kLog2e, -logs);
      const float p = __builtin_amdgcn_exp2f(q);
      float g = -p * __builtin_fmaf(g1, fmaxf(q, -300.f), g0);
      if (empty) g = 0.f;
      if (j + e == t) g += gl;
      d[e] = g;
    }
    store_vec(out, j, V, d, same);
  }
}

namespace {

// The teacher's side of a row.
struct TeacherRow {
  float q[kDistillMax];       // entry's probability; 0 for no entry
  float total[kDistillMax];   // at a word's first entry the sum over its entries, 0 at later ones
  int idx[kDistillMax];       // word; -1 for no entry
  double loss[kDistillMax / 64];
  float top, logsum;
  bool any;
};

// What thread k < K keeps of entry k.
struct Entry {
  int64_t j;     // word as given
  float v;       // the teacher's logit
  float z;       // the student's logit
  double logq;
};

// Entry k's loads, to be issued before the row's: loads come back in order.
__device__ __forceinline__ Entry load_entry(const Teacher &t, int64_t m) {
  const int k = threadIdx.x;
  Entry x{-1, -INFINITY, 0.f, 0.0};
  if (k < t.K) {
    x.j = t.idx[m * t.K + k];
    x.v = t.val[m * t.K + k];
  }
  return x;
}

// Fills sh and the rest of the entry; every thread of the workgroup takes
// part (NT >= K).
template <typename T>
__device__ __forceinline__ void teacher_row(TeacherRow &sh, Entry &x, const T *zrow, int V, const Teacher &t, float c) {
  const int k = threadIdx.x;
  const bool real = k < t.K && x.j >= 0 && x.j < V;
  const int j = real ? static_cast<int>(x.j) : -1;
  if (k < t.K) {
    sh.idx[k] = j;
    sh.q[k] = real ? x.v : -INFINITY;
  }
  if (real) x.z = as_f32(zrow[j]);
  __syncthreads();
  if (k < 64) {   // wave 0: the softmax of the list
    float w[kDistillMax / 64], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kDistillMax / 64; ++i) {
      w[i] = 64 * i + k < t.K ? sh.q[64 * i + k] : -INFINITY;
      top = fmaxf(top, w[i]);
    }
    top = wave_max(top);
    const float a = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < kDistillMax / 64; ++i) {
      w[i] = __builtin_amdgcn_exp2f((w[i] - a) * c);
      sum += w[i];
    }
    sum = wave_sum(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < kDistillMax / 64; ++i)
      if (64 * i + k < t.K) sh.q[64 * i + k] = w[i] * inv;
    if (k == 0) {
      sh.any = sum != 0.f;
      sh.top = top;
      sh.logsum = __builtin_amdgcn_logf(sum) * 0.693147182f;   // v_log_f32: to base 2
    }
  }
  __syncthreads();
  if (k < t.K) {
    float total = 0.f;
    if (real) {
      x.logq = (static_cast<double>(x.v) - static_cast<double>(sh.top)) / static_cast<double>(t.temperature) -
               static_cast<double>(sh.logsum);
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
}

// Sum of q (log q - log p) in a fixed order, in thread 0.
__device__ __forceinline__ double distill_loss(TeacherRow &sh, int K, double logq, double logp) {
  double v = 0.0;
  const int k = threadIdx.x;
  if (k < K && sh.idx[k] >= 0 && sh.q[k] != 0.f) v = static_cast<double>(sh.q[k]) * (logq - logp);
  if (k < kDistillMax) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((k & 63) == 0) sh.loss[k >> 6] = v;
  }
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kDistillMax / 64; ++w) s += sh.loss[w];
  return s;
}

// The listed words' gradients, written over the row's own once every wave's
// stores are acknowledged.
template <typename T>
__device__ __forceinline__ void put_listed(const TeacherRow &sh, int K, float p, float scale, int lo, int hi, T *out) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  const int k = threadIdx.x;
  if (k < K && sh.total[k] != 0.f && scale != 0.f) {
    const int j = sh.idx[k];
    if (j >= lo && j < hi) out[j] = static_cast<T>((p - sh.total[k]) * scale);
  }
}

}  // namespace

// One workgroup: one row, its loss and (kGrad) its gradient.  z is read once:
// the words stay in registers from the maximum to the gradient.  8192 rows of
// 32000 bf16 words 214 to 219 us (4.8 TB/s read and written), 128 rows 11 us.
template <typename T, int NT, bool kGrad>
__global__ __launch_bounds__(NT, kGrad ? (NT == 1024 ? 4 : 6) : 8) void k_distill_row(const T *Z, int V, int64_t ld, int per, float c, Teacher t,
                                                    const float *__restrict__ weight, float *__restrict__ loss,
                                                    float *__restrict__ lse, T *dZ, int64_t ldd) {
  constexpr int n = Words<T>::n;
  __shared__ float sh_max[NT / 64], sh_sum[NT / 64][2];
  __shared__ TeacherRow sh;
  const int64_t m = blockIdx.x;
  const Row<T> row(Z, ld, m, V);
  Entry en = load_entry(t, m);
  Held<T, NT> h;
  h.load(row, 0, per);
  teacher_row(sh, en, row.p, V, t, c);
  float vm[kVecs];
  const float zmax = block_max(h.maximum(vm, per), sh_max);
  const Exps x(zmax, c);
  float s, u;
  block_sums<false>(h, x, per, s, u, sh_sum);
  const Partial p = corrected(x, zmax, s, 0.f);
  if constexpr (kGrad) {
    const bool empty = zmax == -INFINITY && s == 0.f;
    const float w = empty ? 0.f : (weight ? weight[m] : 1.f) / t.temperature;
    const float scale = sh.any ? w : 0.f, f = scale == 0.f ? 0.f : scale / s;
    T *out = dZ + m * ldd;
    const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(row.p) & 15);
    h.again();
    Exps y = x;
    if (scale == 0.f) {   // no gradient, whatever the row holds: 2^0 f = 0
      h.zero();
      y.c = y.r = 0.f;
      y.far = false;
    }
    auto put = [&](auto far) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        if (NT * i >= per) continue;
        const int v = static_cast<int>(threadIdx.x) + NT * i;
        float d[n];
#pragma unroll
        for (int e = 0; e < n; ++e) d[e] = __builtin_amdgcn_exp2f(y.template t<decltype(far)::value>(h.x[i].get(e))) * f;
        if (same && Held<T, NT>::full(row, 0, per, i))
          store_inside(out, row.mis, v, d);
        else if (v < per)
          store_vec(out, row.first(v), V, d, same);
      }
    };
    if (y.far)
      put(std::true_type());
    else
      put(std::false_type());
    const float pk = x.far ? __builtin_amdgcn_exp2f(x.t<true>(en.z)) / s : __builtin_amdgcn_exp2f(x.t<false>(en.z)) / s;
    put_listed(sh, t.K, pk, scale, 0, V, out);
  }
  const RowSums o = row_sums(p.a, p.s, 0.0);
  const double l = distill_loss(sh, t.K, en.logq, log_p(o, en.z, t.temperature));
  if (threadIdx.x == 0) {
    loss[m] = sh.any ? static_cast<float>(l) : 0.f;
    put_lse(lse, m, o);
  }
}

// One workgroup a row, after k_vocab_slice.
template <typename T>
__global__ __launch_bounds__(kDistillMax) void k_distill_join(const T *__restrict__ Z, int V, int64_t ld, int S, float c,
                                                              Teacher t, const Partial *__restrict__ part,
                                                              float *__restrict__ loss, float *__restrict__ lse) {
  __shared__ TeacherRow sh;
  const int64_t m = blockIdx.x;
  Entry en = load_entry(t, m);
  teacher_row(sh, en, Z + m * ld, V, t, c);
  const RowSums o = join(part + m * S, S, c);
  const double l = distill_loss(sh, t.K, en.logq, log_p(o, en.z, t.temperature));
  if (threadIdx.x == 0) {
    loss[m] = sh.any ? static_cast<float>(l) : 0.f;
    put_lse(lse, m, o);
  }
}

// One workgroup: `per` vectors of one row, in steps of kGradVecs.
template <typename T>
__global__ __launch_bounds__(kVThreads) void k_distill_bwd(const T *Z, int V, int64_t ld, int chunks, int per, float c,
                                                           Teacher t, const float *__restrict__ lse,
                                                           const float *__restrict__ weight, T *dZ, int64_t ldd) {
  constexpr int n = Words<T>::n;
  __shared__ TeacherRow sh;
  const int64_t m = blockIdx.x / chunks;
  const int first = static_cast<int>(blockIdx.x % chunks) * per;
  const Row<T> row(Z, ld, m, V);
  T *out = dZ + m * ldd;
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(row.p) & 15);
  Entry en = load_entry(t, m);
  teacher_row(sh, en, row.p, V, t, c);
  const float a = lse[2 * m], logs = lse[2 * m + 1] * kLog2e;
  const bool empty = a == -INFINITY && logs == 0.f;
  const float ref = a == -INFINITY ? 0.f : a;
  const float w = empty ? 0.f : (weight ? weight[m] : 1.f) / t.temperature;
  const float scale = sh.any ? w : 0.f;
  const int end = min(first + per, (V + row.mis + n - 1) / n);
  for (int v0 = first; v0 < end; v0 += kGradVecs) {
#pragma unroll
    for (int i = 0; i < kGradVecs / kVThreads; ++i) {
      const int v = v0 + static_cast<int>(threadIdx.x) + kVThreads * i;
      if (v >= end) break;
      const Words<T> x = row.load(v);
      float d[n];
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(x.get(e) - ref, c, -logs));
        d[e] = scale == 0.f ? 0.f : p * scale;
      }
      store_vec(out, row.first(v), V, d, same);
    }
  }
  put_listed(sh, t.K, __builtin_amdgcn_exp2f(__builtin_fmaf(en.z - ref, c, -logs)), scale, max(row.first(first), 0),
             min(row.first(first + per), V), out);
}

namespace {

template <typename T>
int row_vecs(int64_t V) {
  return static_cast<int>((V + 2 * Words<T>::n - 2) / Words<T>::n);
}

template <typename T>
int grad_chunks(int64_t V) {
  return (row_vecs<T>(V) + kGradVecs - 1) / kGradVecs;
}

float scaled_log2e(float temperature) {
  return static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
}

template <typename T, bool kEntropy, bool kTop>
hipError_t launch_slice(const Logits &l, const Slices &sl, float c, int top, Partial *part, uint64_t *keys, hipStream_t s) {
  hipLaunchKernelGGL((k_vocab_slice<T, kEntropy, kTop>), dim3(static_cast<uint32_t>(l.M * sl.S)), dim3(kVThreads), 0, s,
                     static_cast<const T *>(l.z), static_cast<int>(l.V), l.ld, sl.S, sl.per, c, top, part, keys);
  return hipGetLastError();
}

template <typename T, bool kTop>
hipError_t logprobs_as(const Logits &l, const int64_t *target, int top, const LogprobOut &out, void *ws, hipStream_t s) {
  const Slices sl = slices_of(l, top);
  const T *z = static_cast<const T *>(l.z);
  const int V = static_cast<int>(l.V);
  const dim3 rows(static_cast<uint32_t>(l.M));
  if (sl.S == 1) {
    if (sl.threads == 256)
      hipLaunchKernelGGL((k_logprobs_row<T, 256, kTop>), rows, dim3(256), 0, s, z, V, l.ld, sl.per, target, top, out);
    else if (sl.threads == 512)
      hipLaunchKernelGGL((k_logprobs_row<T, 512, kTop>), rows, dim3(512), 0, s, z, V, l.ld, sl.per, target, top, out);
    else
      hipLaunchKernelGGL((k_logprobs_row<T, 1024, kTop>), rows, dim3(1024), 0, s, z, V, l.ld, sl.per, target, top, out);
    return hipGetLastError();
  }
  Partial *part = static_cast<Partial *>(ws);
  uint64_t *keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) +
                                                up256(static_cast<size_t>(l.M) * sl.S * sizeof(Partial)));
  const hipError_t e = launch_slice<T, true, kTop>(l, sl, kLog2e, top, part, keys, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_logprobs_join<T, kTop>), rows, dim3(kTop ? kVThreads : 64), 0, s, z, V, l.ld, sl.S, target, top,
                     part, keys, out);
  return hipGetLastError();
}

template <typename T>
hipError_t logprobs_bwd_as(const Logits &l, const int64_t *target, const float *lse, const float *entropy,
                           const float *g_logprob, const float *g_entropy, void *dz, int64_t ldd, hipStream_t s) {
  const int chunks = grad_chunks<T>(l.V);
  hipLaunchKernelGGL(k_logprobs_bwd<T>, dim3(static_cast<uint32_t>(l.M * chunks)), dim3(kVThreads), 0, s,
                     static_cast<const T *>(l.z), static_cast<int>(l.V), l.ld, chunks, target, lse, entropy, g_logprob,
                     g_entropy, static_cast<T *>(dz), ldd);
  return hipGetLastError();
}

template <typename T, bool kGrad>
hipError_t distill_row_as(const Logits &l, const Teacher &t, const Slices &sl, const float *weight, float *loss, float *lse,
                          void *dz, int64_t ldd, hipStream_t s) {
  const T *z = static_cast<const T *>(l.z);
  T *d = static_cast<T *>(dz);
  const int V = static_cast<int>(l.V);
  const dim3 rows(static_cast<uint32_t>(l.M));
  const float c = scaled_log2e(t.temperature);
  if (sl.threads == 256)
    hipLaunchKernelGGL((k_distill_row<T, 256, kGrad>), rows, dim3(256), 0, s, z, V, l.ld, sl.per, c, t, weight, loss, lse, d,
                       ldd);
  else if (sl.threads == 512)
    hipLaunchKernelGGL((k_distill_row<T, 512, kGrad>), rows, dim3(512), 0, s, z, V, l.ld, sl.per, c, t, weight, loss, lse, d,
                       ldd);
  else
    hipLaunchKernelGGL((k_distill_row<T, 1024, kGrad>), rows, dim3(1024), 0, s, z, V, l.ld, sl.per, c, t, weight, loss, lse,
                       d, ldd);
  return hipGetLastError();
}

template <typename T>
hipError_t distill_fwd_as(const Logits &l, const Teacher &t, float *loss, float *lse, void *ws, hipStream_t s) {
  const Slices sl = slices_of(l, 0);
  if (sl.S == 1) return distill_row_as<T, false>(l, t, sl, nullptr, loss, lse, nullptr, 0, s);
  const float c = scaled_log2e(t.temperature);
  Partial *part = static_cast<Partial *>(ws);
  const hipError_t e = launch_slice<T, false, false>(l, sl, c, 0, part, nullptr, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_distill_join<T>, dim3(static_cast<uint32_t>(l.M)), dim3(kDistillMax), 0, s,
                     static_cast<const T *>(l.z), static_cast<int>(l.V), l.ld, sl.S, c, t, part, loss, lse);
  return hipGetLastError();
}

// Steps of kGradVecs vectors of a workgroup: the teacher's list is worked out
// once in each, so the whole row, down to one step where there are few rows.
template <typename T>
int distill_steps(int64_t M, int64_t V) {
  const int most = grad_chunks<T>(V);
  const int64_t want = std::min<int64_t>(most, std::max<int64_t>(1, 2048 / M));
  return static_cast<int>((most + want - 1) / want);
}

template <typename T>
hipError_t distill_bwd_as(const Logits &l, const Teacher &t, const float *lse, const float *weight, void *dz,
                          int64_t ldd, hipStream_t s) {
  const int steps = distill_steps<T>(l.M, l.V), chunks = (grad_chunks<T>(l.V) + steps - 1) / steps;
  hipLaunchKernelGGL(k_distill_bwd<T>, dim3(static_cast<uint32_t>(l.M * chunks)), dim3(kVThreads), 0, s,
                     static_cast<const T *>(l.z), static_cast<int>(l.V), l.ld, chunks, steps * kGradVecs,
                     scaled_log2e(t.temperature), t, lse, weight, static_cast<T *>(dz), ldd);
  return hipGetLastError();
}

template <typename T>
hipError_t distill_as(const Logits &l, const Teacher &t, const float *weight, float *loss, float *lse, void *dz, int64_t ldd,
                      void *ws, hipStream_t s) {
  const Slices sl = slices_of(l, 0);
  if (sl.S == 1) return distill_row_as<T, true>(l, t, sl, weight, loss, lse, dz, ldd, s);
  const hipError_t e = distill_fwd_as<T>(l, t, loss, lse, ws, s);
  return e != hipSuccess ? e : distill_bwd_as<T>(l, t, lse, weight, dz, ldd, s);
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
  const LogprobOut out{logprob, entropy, lse, top_logprob, top_index};
  QLORA_BY_TYPE(l.type, (top ? logprobs_as<T, true>(l, target, top, out, ws, s)
                             : logprobs_as<T, false>(l, target, top, out, ws, s)))
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
  QLORA_BY_TYPE(l.type, distill_as<T>(l, t, weight, loss, lse, dz, ldd, ws, s))
}

int64_t vocab_row_threads(int64_t M, int64_t V, int type, int top) {
  const Slices a = slices_of(M, V, type, top, true), b = slices_of(M, V, type, top, false);
  return std::max(int64_t{a.S} * a.threads, int64_t{b.S} * b.threads);
}

int64_t logprobs_bwd_row_threads(int64_t V, int type) {
  QLORA_BY_TYPE(type, int64_t{grad_chunks<T>(V)} * kVThreads)
}

int64_t distill_bwd_row_threads(int64_t M, int64_t V, int type) {
  QLORA_BY_TYPE(type, int64_t{(grad_chunks<T>(V) + distill_steps<T>(M, V) - 1) / distill_steps<T>(M, V)} * kVThreads)
}

#undef QLORA_BY_TYPE

}  // namespace qlora
