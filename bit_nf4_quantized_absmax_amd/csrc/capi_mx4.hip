// C ABI of the MX4 codec and the linear layer on MX4 weights: argument
// validation, workspace carving and the composite passes.  Every check runs
// before anything is launched.
#include <math.h>

#include <algorithm>

#include "capi_util.h"

using namespace qlora;

namespace {

constexpr int64_t kMaxCols = int64_t{1} << 24;   // 256 rows of codes stay within 32-bit offsets

// Rows and columns of an MX4 array; rows = 0 (no tokens) only where allowed.
int check_mx4_shape(int64_t rows, int64_t cols, bool empty_ok) {
  if (rows < (empty_ok ? 0 : 1) || cols < 1) return QLORA_ERR_INVALID_ARG;
  if (cols % 32 != 0 || rows > kMaxElems || cols > kMaxCols) return QLORA_ERR_UNSUPPORTED_SHAPE;
  return QLORA_OK;
}

int check_mx4(const qlora_mx4_array *a, bool empty_ok) {
  if (!a) return QLORA_ERR_INVALID_ARG;
  const int st = check_mx4_shape(a->rows, a->cols, empty_ok);
  if (st) return st;
  if (!rows_ok(a->codes, a->rows) || !rows_ok(a->scales, a->rows)) return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

Mx4View view_of(const qlora_mx4_array *a) { return Mx4View{a->codes, a->scales, a->rows, a->cols}; }

size_t code_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * mx4_slabs(cols) * 128; }
size_t scale_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * mx4_slabs(cols) * 8; }

// Shape rules of a product and of the linear layer: the arrays' for X and W, an
// optional LoRA pair of rank r (0: none) and the LoRA kernels' size limit with it.
int check_shape(int64_t M, int64_t N, int64_t K, int32_t r, bool bwd) {
  if (M < 0) return QLORA_ERR_INVALID_ARG;
  int st = check_mx4_shape(N, K, false);
  if (!st) st = check_mx4_shape(M, K, true);
  if (st) return st;
  if (r < 0 || r > 128 || (bwd && r < 1)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (bwd && (K % 64 != 0 || N % 8 != 0 || N > kMaxElems / K)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if ((M + 127) / 128 * ((N + 127) / 128) > kMaxElems) return QLORA_ERR_UNSUPPORTED_SHAPE;   // the product's tiles
  if (mx4_small_ok(M) && !mx4_small_launch_ok(N)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (r > 0 && M > 0 && M > kMaxElems / std::max(N, K)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  return QLORA_OK;
}

// The linear layer's: X is rounded here.
int check_linear(int64_t M, int64_t N, int64_t K, int32_t r, bool bwd) {
  const int st = check_shape(M, N, K, r, bwd);
  return st || mx4_quantize_ok(M, K) ? st : QLORA_ERR_UNSUPPORTED_SHAPE;
}

// How T and X's rounding are made above the decode sizes, by measurement (us,
// both):              partial sums   LoRA product and codec   one pass
//   75 x 8224, r 64         8.9               26.4               40.4
//   512 x 4096, r 64       12.3               14.3               26.0
//   1024 x 4096, r 64      15.7               14.7               26.2
//   1536 x 4096, r 64      19.9               15.1               26.7
//   1536 x 4096, r 8       12.2               14.8               14.7
//   8192 x 4096, r 8                          31.2               23.2
// Partial sums fetch X once per 16 adapter rows, and win while tokens times
// such tiles are 4096 at most; from 2048 tokens on, one pass for a single tile.
bool by_partials(int64_t M, int32_t r) {
  return r > 0 && (mx4_small_ok(M) || (M < 2048 && M * ((r + 15) / 16) <= 4096));
}

// Workspace of the forward pass: T (when the caller keeps none) | partial sums
// of T | X's codes | X's scales | the product's split tiles.
struct FwdWs {
  size_t t, p, codes, scales, total;
};
FwdWs fwd_ws(int64_t M, int64_t N, int64_t K, int32_t r) {
  FwdWs w;
  w.t = mx4_small_ok(M) ? 0 : bf16_bytes(M * r);
  w.p = by_partials(M, r) ? round_up(mx4_small_ws_bytes(M, K, r), 256) : 0;
  w.codes = round_up(code_bytes(M, K), 256);
  w.scales = round_up(scale_bytes(M, K), 256);
  w.total = w.t + w.p + w.codes + w.scales + (mx4_small_ok(M) ? 0 : mx4_split_ws_bytes(M, N, K));
  return w;
}

// Workspace of a dX of few tiles, after the others: A^T | partial tiles.
struct DxWs {
  size_t at, total;
};
DxWs dx_ws(int64_t M, int64_t N, int64_t K, int32_t r) {
  if (N % 64 != 0 || !mx4_dx_small_ok(M, N, K)) return DxWs{0, 0};
  const size_t at = bf16_bytes(K * r);
  return DxWs{at, at + mx4_dx_small_ws_bytes(M, N, K)};
}

}  // namespace

extern "C" {

int qlora_mx4_sizes(int64_t rows, int64_t cols, int64_t *codes, int64_t *scales) {
  const int st = check_mx4_shape(rows, cols, true);
  if (st) return st;
  if (codes) *codes = static_cast<int64_t>(code_bytes(rows, cols));
  if (scales) *scales = static_cast<int64_t>(scale_bytes(rows, cols));
  return QLORA_OK;
}

int qlora_mx4_quantize(const void *X, int32_t in_type, const qlora_mx4_array *out, void *stream) {
  const int st = check_mx4(out, true);
  if (st) return st;
  if (!mx4_quantize_ok(out->rows, out->cols)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (in_type < 0 || in_type > QLORA_IN_FP16 || !rows_ok(X, out->rows)) return QLORA_ERR_INVALID_ARG;
  if (out->rows == 0) return QLORA_OK;
  return from_hip(launch_mx4_quantize(X, in_type, view_of(out), static_cast<hipStream_t>(stream)));
}

int qlora_mx4_dequantize(const qlora_mx4_array *a, uint16_t *out_bf16, void *stream) {
  const int st = check_mx4(a, true);
  if (st) return st;
  if (!mx4_dequantize_ok(a->rows, a->cols)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (!rows_ok(out_bf16, a->rows)) return QLORA_ERR_INVALID_ARG;
  if (a->rows == 0) return QLORA_OK;
  return from_hip(launch_mx4_dequantize(view_of(a), out_bf16, static_cast<hipStream_t>(stream)));
}

int qlora_mx4_matmul(const qlora_mx4_array *X, const qlora_mx4_array *W, const uint16_t *T, const uint16_t *B, int32_t r,
                     uint16_t *Y, void *stream) {
  int st = check_mx4(X, true);
  if (!st) st = check_mx4(W, false);
  if (st) return st;
  if (X->cols != W->cols) return QLORA_ERR_INVALID_ARG;
  st = check_shape(X->rows, W->rows, W->cols, r, false);
  if (st) return st;
  if (!rows_ok(Y, X->rows) || (r > 0 && (!rows_ok(T, X->rows) || !bf16_ok(B)))) return QLORA_ERR_INVALID_ARG;
  if (X->rows == 0) return QLORA_OK;
  if (mx4_small_ok(X->rows))
    return from_hip(launch_mx4_small_matmul(view_of(X), view_of(W), T, B, r, Y, static_cast<hipStream_t>(stream)));
  return from_hip(launch_mx4_matmul(view_of(X), view_of(W), T, B, r, Y, nullptr, static_cast<hipStream_t>(stream)));
}

size_t qlora_mx4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t r, int is_bwd) {
  if (M == 0 || check_linear(M, N, K, r, is_bwd != 0)) return 0;
  if (!is_bwd) return fwd_ws(M, N, K, r).total;
  return bf16_bytes(N * K) + bwd_ws(M, N, K, r).total + dx_ws(M, N, K, r).total;
}

int qlora_mx4_linear_fwd(const uint16_t *X, int64_t M, const qlora_mx4_array *W, const uint16_t *A, const uint16_t *B,
                         int32_t r, float scale, uint16_t *Y, uint16_t *T_out, void *ws, size_t ws_bytes, void *stream) {
  int st = check_mx4(W, false);
  if (!st) st = check_linear(M, W->rows, W->cols, r, false);
  if (st) return st;
  if (!rows_ok(X, M) || !rows_ok(Y, M)) return QLORA_ERR_INVALID_ARG;
  if (r > 0 && (!bf16_ok(A) || !bf16_ok(B) || !bf16_opt(T_out) || !isfinite(scale))) return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  const FwdWs L = fwd_ws(M, W->rows, W->cols, r);
  if (!ws || !aligned(ws, 16) || ws_bytes < L.total) return QLORA_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t *base = static_cast<uint8_t *>(ws);
  float *P = reinterpret_cast<float *>(base + L.t);
  uint8_t *codes = base + L.t + L.p;
  const Mx4View x{codes, codes + L.codes, M, W->cols};
  if (mx4_small_ok(M))
    return from_hip(launch_mx4_small_linear(X, view_of(W), A, B, r, scale, Y, r > 0 ? T_out : nullptr, P, x, s));
  uint16_t *T = r > 0 && T_out ? T_out : reinterpret_cast<uint16_t *>(base);
  hipError_t e = hipSuccess;
  if (by_partials(M, r)) {
    e = launch_mx4_prep(X, x, A, r, scale, T, P, s);
  } else if (r > 0 && r <= kMx4RowsMax) {
    e = launch_mx4_rows(X, x, A, r, scale, T, s);
  } else {
    if (r > 0) e = launch_lora_down(X, static_cast<int>(M), static_cast<int>(W->cols), A, r, scale, T, s);
    if (e == hipSuccess) e = launch_mx4_quantize(X, QLORA_IN_BF16, x, s);
  }
  if (e != hipSuccess) return QLORA_ERR_HIP;
  return from_hip(launch_mx4_matmul(x, view_of(W), T, B, r, Y, codes + L.codes + L.scales, s));
}

int qlora_mx4_linear_bwd(const uint16_t *dY, const uint16_t *X, const uint16_t *T, int64_t M, const qlora_mx4_array *W,
                         const uint16_t *A, const uint16_t *B, int32_t r, float scale, uint16_t *dX, uint16_t *dA,
                         uint16_t *dB, void *ws, size_t ws_bytes, void *stream) {
  int st = check_mx4(W, false);
  if (!st) st = check_linear(M, W->rows, W->cols, r, true);
  if (st) return st;
  if (dX && W->rows % 64 != 0) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (!rows_ok(dY, M) || !rows_ok(X, M) || !bf16_ok(A) || !bf16_ok(B) || !isfinite(scale)) return QLORA_ERR_INVALID_ARG;
  if (!bf16_opt(T) || !bf16_opt(dX) || !bf16_opt(dA) || !bf16_opt(dB)) return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  const int64_t N = W->rows, K = W->cols;
  const BwdWs L = bwd_ws(M, N, K, r);
  const size_t wd_bytes = bf16_bytes(N * K);
  const DxWs D = dx_ws(M, N, K, r);
  if (!ws || !aligned(ws, 16) || ws_bytes < wd_bytes + L.total + D.total) return QLORA_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
  uint16_t *Wd = static_cast<uint16_t *>(ws);
  char *base = static_cast<char *>(ws) + wd_bytes;
  uint16_t *Tw = reinterpret_cast<uint16_t *>(base);
  uint16_t *G = reinterpret_cast<uint16_t *>(base + L.t);
  void *bt = base + L.t + L.g;
  void *pa = base + L.t + L.g + L.bt;
  void *pb = base + L.t + L.g + L.bt + L.pa;
  if ((dX || dA) && launch_lora_grad_in(dY, m, n, B, r, scale, G, bt, s) != hipSuccess) return QLORA_ERR_HIP;
  if (dX && D.total > 0) {
    uint16_t *At = reinterpret_cast<uint16_t *>(base + L.total);
    if (launch_mx4_transpose(view_of(W), A, r, Wd, At, s) != hipSuccess) return QLORA_ERR_HIP;
    if (launch_mx4_dx_small(dY, Wd, G, At, m, n, k, r, dX, base + L.total + D.at, s) != hipSuccess) return QLORA_ERR_HIP;
  } else if (dX) {
    if (launch_mx4_dequantize(view_of(W), Wd, s) != hipSuccess) return QLORA_ERR_HIP;
    const NF4View shape{nullptr, nullptr, nullptr, nullptr, n, k, 0};
    if (launch_pre_matmul_dx(MatmulJob{dY, G, A, nullptr, dX, shape, m, r, Wd}, s) != hipSuccess) return QLORA_ERR_HIP;
  }
  const uint16_t *Tu = T;
  if (dB && !Tu) {
    if (launch_lora_down(X, m, k, A, r, scale, Tw, s) != hipSuccess) return QLORA_ERR_HIP;
    Tu = Tw;
  }
  const int sp = lora_grad_splits(m, k, n, r, dA != nullptr, dB != nullptr);
  GradWJob jobs[2];
  int nj = 0;
  if (dA) jobs[nj++] = GradWJob{X, G, m, k, r, true, dA, pa, sp};
  if (dB) jobs[nj++] = GradWJob{dY, Tu, m, n, r, false, dB, pb, sp};
  if (nj > 0 && launch_lora_grad_w_group(nj, jobs, s) != hipSuccess) return QLORA_ERR_HIP;
  return QLORA_OK;
}

}  // extern "C"
