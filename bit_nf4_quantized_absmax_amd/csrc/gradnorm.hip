// The norm of a model's gradients and clipping by it (gfx950), over any number
// of tensors:
//     norm_g = sqrt(sum of x^2 over the elements of group g)
//     out    = x min(1, max_norm / (norm_g + 1e-6))
// Every tensor is `groups` equal parts along its first axis, part g of group g
// (groups = 1: one norm of all; groups = n: one for each of n adapters whose
// gradients are stacked).
//
//  * Bound by reading the gradients twice and writing them once; the second
//    read comes from the memory-side cache while they fit there (256 MB).  448 tensors, 320
//    MB: 106 us for the squares in four launches, whose starts and ends cost a third of
//    it (18 to 29 us each for 80 MB), and 115 for the clipping (5.6 TB/s read and
//    written); larger chunks, more of them and more loads at once were the same.  14
//    small tensors: 4 + 4.  Around them the host's walk over the list takes 0.5 us a tensor, and
//    telling autograd of the change 0.03.
//  * Squares are summed in 64 bits: no size of finite gradients overflows, and
//    the order of the sums shows in the last bits of fp32 at most.  An fp64
//    multiply-add a value keeps up with the stream (4 T of either a second).
//  * A workgroup takes a chunk of one part of one tensor and leaves one partial
//    sum; the order of all sums is fixed, so results repeat.  The list of
//    tensors is an argument of the launch that sums them (kGradList of them, one
//    launch after the other), which also writes the table of chunks that the
//    clipping kernel reads: nothing is copied from the host.
//  * The clipping kernel's workgroups each add up their group's partial sums
//    (about 2000, from L2): one launch less.  A list of far more tensors than 2000 has as many
//    chunks, and pays the square of their number in reads from L2.  Where nothing has to change and the
//    result goes where it came from, a workgroup ends there.
#include <algorithm>

#include "common.h"
#include "launch.h"

namespace qlora {

namespace {

constexpr int kGnThreads = 256;

template <class T>
__device__ __forceinline__ float value(T v);
template <>
__device__ __forceinline__ float value(float v) { return v; }
template <>
__device__ __forceinline__ float value(uint16_t v) { return bf16_to_f32(v); }
template <>
__device__ __forceinline__ float value(_Float16 v) { return static_cast<float>(v); }

template <class T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t narrow(float v) { return f32_to_bf16(v); }
template <>
__device__ __forceinline__ _Float16 narrow(float v) { return static_cast<_Float16>(v); }

template <class T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
  T v[n];
};

__device__ __forceinline__ double block_sum(double v, double *sh) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kGnThreads / 64; ++w) t += sh[w];
  __syncthreads();
  return t;
}

template <class T>
__device__ __forceinline__ double squares(const T *x, int64_t count) {
  constexpr int n = Vec<T>::n;
  // up to the first 16-byte boundary and after the last whole one: single elements
  const int head = static_cast<int>(min(count, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T))));
  double s = 0.0;
  if (static_cast<int>(threadIdx.x) < head) {
    const double v = value(x[threadIdx.x]);
    s = v * v;
  }
  const Vec<T> *xv = reinterpret_cast<const Vec<T> *>(x + head);
  const int64_t whole = (count - head) / n;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < whole; i += kGnThreads) {
    const Vec<T> v = xv[i];
#pragma unroll
    for (int e = 0; e < n; ++e) {
      const double d = value(v.v[e]);
      s = __builtin_fma(d, d, s);
    }
  }
  const int64_t rest = head + whole * n + threadIdx.x;
  if (rest < count) {
    const double v = value(x[rest]);
    s = __builtin_fma(v, v, s);
  }
  return s;
}

// Times c in two steps: a factor below fp32's normal range (a norm above 2^100)
// would lose its last bits.
struct Factor {
  float pre, c;
  __device__ __forceinline__ explicit Factor(double v) : pre(v < 0x1p-100 ? 0x1p-64f : 1.f), c(static_cast<float>(v / pre)) {}
  __device__ __forceinline__ float operator()(float x) const { return x * pre * c; }
};

template <class T>
__device__ __forceinline__ void scaled(const T *x, T *y, int64_t count, Factor f) {
  constexpr int n = Vec<T>::n;
  if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15) != 0) {   // no common 16-byte boundary
    for (int64_t i = threadIdx.x; i < count; i += kGnThreads) y[i] = narrow<T>(f(value(x[i])));
    return;
  }
  const int head = static_cast<int>(min(count, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T))));
  if (static_cast<int>(threadIdx.x) < head) y[threadIdx.x] = narrow<T>(f(value(x[threadIdx.x])));
  const Vec<T> *xv = reinterpret_cast<const Vec<T> *>(x + head);
  Vec<T> *yv = reinterpret_cast<Vec<T> *>(y + head);
  const int64_t whole = (count - head) / n;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < whole; i += kGnThreads) {
    Vec<T> v = xv[i];
#pragma unroll
    for (int e = 0; e < n; ++e) v.v[e] = narrow<T>(f(value(v.v[e])));
    yv[i] = v;
  }
  const int64_t rest = head + whole * n + threadIdx.x;
  if (rest < count) y[rest] = narrow<T>(f(value(x[rest])));
}

}  // namespace

// One list's chunks: workgroup (group, chunk of the list's share of a group) finds its
// tensor, writes its entry of the table and its sum of squares.
__global__ __launch_bounds__(kGnThreads) void k_grad_squares(const GradList l, GradPlan p, int lead) {
  __shared__ double sh[kGnThreads / 64];
  const int g = blockIdx.x / l.chunks, c = l.t[0].first + blockIdx.x % l.chunks;
  int lo = 0, hi = l.n - 1;                      // the last tensor whose first chunk is not behind this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.t[mid].first <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  const GradTensor t = l.t[lo];
  const int64_t part = t.part, in = static_cast<int64_t>(c - t.first) * p.chunk;
  const int64_t at = g * part + in;
  const int count = static_cast<int>(min(static_cast<int64_t>(p.chunk), part - in));
  const int64_t place = static_cast<int64_t>(g) * p.stride + c;
  if (threadIdx.x == 0 && t.y) {
    const int64_t bytes = at * (t.type == 0 ? 4 : 2);
    p.table[place] = GradChunk{static_cast<const char *>(t.x) + bytes, static_cast<char *>(t.y) + bytes, count, t.type, g,
                               lead && c == 0 ? 1 : 0};
  }
  double s;
  if (t.type == 0)
    s = squares(static_cast<const float *>(t.x) + at, count);
  else if (t.type == 1)
    s = squares(static_cast<const uint16_t *>(t.x) + at, count);
  else
    s = squares(static_cast<const _Float16 *>(t.x) + at, count);
  s = block_sum(s, sh);
  if (threadIdx.x == 0) p.sums[place] = s;
}

__device__ __forceinline__ double group_norm(const GradPlan &p, int group, double *sh) {
  double s = 0.0;
  for (int i = threadIdx.x; i < p.stride; i += kGnThreads) s += p.sums[static_cast<int64_t>(group) * p.stride + i];
  return sqrt(block_sum(s, sh));
}

__global__ __launch_bounds__(kGnThreads) void k_grad_norm(GradPlan p, float *__restrict__ norm) {
  __shared__ double sh[kGnThreads / 64];
  const double n = group_norm(p, blockIdx.x, sh);
  if (threadIdx.x == 0) norm[blockIdx.x] = static_cast<float>(n);
}

__global__ __launch_bounds__(kGnThreads) void k_grad_clip(GradPlan p, float max_norm, float *__restrict__ norm) {
  __shared__ double sh[kGnThreads / 64];
  const GradChunk k = p.table[blockIdx.x];
  const double n = group_norm(p, k.group, sh);
  if (k.lead && threadIdx.x == 0) norm[k.group] = static_cast<float>(n);
  const double c = max_norm / (n + 1e-6);
  if (c >= 1.0 && k.x == k.y) return;
  const Factor f(c >= 1.0 ? 1.0 : c);            // NaN stays
  if (k.type == 0)
    scaled(static_cast<const float *>(k.x), static_cast<float *>(k.y), k.count, f);
  else if (k.type == 1)
    scaled(static_cast<const uint16_t *>(k.x), static_cast<uint16_t *>(k.y), k.count, f);
  else
    scaled(static_cast<const _Float16 *>(k.x), static_cast<_Float16 *>(k.y), k.count, f);
}

// ---------------------------------------------------------------------------
hipError_t launch_grad_squares(const GradList &l, const GradPlan &p, bool lead, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_squares, dim3(l.chunks * p.groups), dim3(kGnThreads), 0, s, l, p, lead ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const GradPlan &p, const float *max_norm, float *norm, hipStream_t s) {
  if (max_norm && p.stride > 0)
    hipLaunchKernelGGL(k_grad_clip, dim3(p.stride * p.groups), dim3(kGnThreads), 0, s, p, *max_norm, norm);
  else
    hipLaunchKernelGGL(k_grad_norm, dim3(p.groups), dim3(kGnThreads), 0, s, p, norm);
  return hipGetLastError();
}

}  // namespace qlora
