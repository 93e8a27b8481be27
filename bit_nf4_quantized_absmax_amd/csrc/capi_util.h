// Argument checks and size arithmetic shared by the C ABI's entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/qlora.h"
#include "launch.h"

namespace qlora {

constexpr int64_t kMaxElems = (int64_t{1} << 31) - 1;  // kernels index rows * cols in int32 where safe

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool bf16_ok(const void *p) { return p && aligned(p, 16); }

inline bool bf16_opt(const void *p) { return !p || aligned(p, 16); }

// A tensor with M rows: at M = 0 it has no storage and its pointer may be NULL.
inline bool rows_ok(const void *p, int64_t M) { return M == 0 ? bf16_opt(p) : bf16_ok(p); }

inline int from_hip(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }

inline size_t bf16_bytes(int64_t n) { return round_up(static_cast<size_t>(n) * 2, 256); }

// Workspace of the backward pass: T (recompute) | G | B^T | dA partials | dB partials.
struct BwdWs {
  size_t t, g, bt, pa, pb, total;
};
inline BwdWs bwd_ws(int64_t M, int64_t N, int64_t K, int32_t r) {
  BwdWs w;
  w.t = bf16_bytes(M * r);
  w.g = bf16_bytes(M * r);
  w.bt = lora_grad_in_ws_bytes(static_cast<int>(N), r);
  const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
  w.pa = round_up(lora_grad_pair_ws_bytes(m, k, k, n, r), 256);
  w.pb = round_up(lora_grad_pair_ws_bytes(m, n, k, n, r), 256);
  w.total = w.t + w.g + w.bt + w.pa + w.pb;
  return w;
}

// The parts of a workspace, in order, each on 256 bytes.
struct Carve {
  char *base;
  size_t used = 0;
  explicit Carve(void *p) : base(static_cast<char *>(p)) {}
  template <class T>
  T *take(size_t n) {
    T *p = reinterpret_cast<T *>(base + used);
    used += round_up(n * sizeof(T), 256);
    return p;
  }
};

}  // namespace qlora
