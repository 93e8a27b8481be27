// C ABI of the linear layer with many adapters: argument validation, workspace
// carving and the composite passes.  Every check runs before anything is launched.
#include <algorithm>

#include "capi_util.h"

using namespace qlora;

namespace {

int check_adapters(int64_t M, const qlora_nf4_weight *W, const qlora_adapters *ad) {
  if (!W || !ad || M < 0) return QLORA_ERR_INVALID_ARG;
  if (!W->packed || !W->code8 || !W->c2 || !W->mean || W->rows < 1 || W->cols < 1) return QLORA_ERR_INVALID_ARG;
  if (!aligned(W->packed, 16) || !aligned(W->code8, 4) || !aligned(W->c2, 4) || !aligned(W->mean, 4)) return QLORA_ERR_INVALID_ARG;
  if (W->qtype < QLORA_Q4_NF4 || W->qtype > QLORA_Q4_INT4) return QLORA_ERR_INVALID_ARG;
  if (ad->count < 1 || ad->r < 1) return QLORA_ERR_INVALID_ARG;
  if (!bf16_ok(ad->A) || !bf16_ok(ad->B) || !ad->scale || !aligned(ad->scale, 4)) return QLORA_ERR_INVALID_ARG;
  if ((M > 0 && !ad->index) || !aligned(ad->index, 8)) return QLORA_ERR_INVALID_ARG;
  const int64_t N = W->rows, K = W->cols;
  if (K % 64 != 0 || N % 8 != 0 || N > kMaxElems / K) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (ad->count > kAdMax || ad->r > 128 || ad->r % 8 != 0) return QLORA_ERR_UNSUPPORTED_SHAPE;
  // 32-bit byte offsets into X, dY and one adapter
  if (std::max<int64_t>(M, ad->r) > kMaxElems / std::max<int64_t>(round_up(N, 64), K)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  return QLORA_OK;
}

NF4View view_of(const qlora_nf4_weight *w) {
  return NF4View{w->packed, w->code8, w->c2, w->mean, static_cast<int>(w->rows), static_cast<int>(w->cols),
                 static_cast<int>(w->qtype)};
}

AdapterSet set_of(const qlora_adapters *a) { return AdapterSet{a->A, a->B, a->scale, a->index, a->count, a->r}; }

AdPlan take_plan(Carve &c, int64_t M, int64_t n) {
  AdPlan p;
  p.perm = c.take<int>(M);
  p.who = c.take<int>(M);
  p.seg = c.take<int>(n + 1);
  p.tile = c.take<int4>(ad_tiles_max(M, n));
  p.ntile = c.take<int>(1);
  p.zero = c.take<uint16_t>(64);
  return p;
}

// Forward: T (when the caller keeps none) | the decoding kernels' sums, or above
// their sizes the order of the tokens, the dequantized weight and T's partial sums.
struct FwdParts {
  uint16_t *T, *Wd;
  char *sums;
  float *part, *tiles;
  AdPlan plan;
};
size_t carve_fwd(void *ws, int64_t M, int64_t N, int64_t K, int32_t n, int32_t r, FwdParts *f) {
  Carve c(ws);
  f->T = c.take<uint16_t>(M * r);
  if (M > kAdSmall) {
    f->plan = take_plan(c, M, n);
    f->Wd = c.take<uint16_t>(N * K);
    f->part = c.take<float>(ad_down_splits(M, K, n) * M * r);
    f->tiles = c.take<float>(ad_matmul_part_floats(M, N, K));
  } else {
    f->sums = c.take<char>(ad_small_ws_bytes(static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), r));
  }
  return c.used;
}

// Backward, with Np = N filled up to 64: T (recomputed) | G | their partial sums | the order | W |
// A transposed | B transposed | dY with filled rows (where Np > N) | split tiles.
struct BwdParts {
  uint16_t *T, *G, *Wd, *At, *Bt, *dYp;
  float *part, *tiles;
  AdPlan plan;
};
size_t carve_bwd(void *ws, int64_t M, int64_t N, int64_t K, int32_t n, int32_t r, BwdParts *b) {
  const int64_t Np = round_up(N, 64);
  Carve c(ws);
  b->T = c.take<uint16_t>(M * r);
  b->G = c.take<uint16_t>(M * r);
  b->part = c.take<float>(std::max(ad_down_splits(M, K, n), ad_down_splits(M, Np, n)) * M * r);
  b->plan = take_plan(c, M, n);
  b->Wd = c.take<uint16_t>(N * K);
  b->At = c.take<uint16_t>(static_cast<int64_t>(n) * r * K);
  b->Bt = c.take<uint16_t>(static_cast<int64_t>(n) * r * Np);
  b->dYp = c.take<uint16_t>(Np > N ? M * Np : 0);
  b->tiles = c.take<float>(ad_matmul_part_floats(M, K, Np));
  return c.used;
}

}  // namespace

extern "C" {

size_t qlora_adapter_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t count, int32_t r, int is_bwd) {
  if (M < 1 || N < 1 || K < 1 || count < 1 || count > kAdMax || r < 8 || r > 128 || r % 8 != 0) return 0;
  if (K % 64 != 0 || N % 8 != 0 || N > kMaxElems / K || std::max<int64_t>(M, r) > kMaxElems / std::max<int64_t>(round_up(N, 64), K))
    return 0;
  FwdParts f;
  BwdParts b;
  return is_bwd ? carve_bwd(nullptr, M, N, K, count, r, &b) : carve_fwd(nullptr, M, N, K, count, r, &f);
}

int qlora_adapter_linear_fwd(const uint16_t *X, int64_t M, const qlora_nf4_weight *W, const qlora_adapters *ad, uint16_t *Y,
                             uint16_t *T_out, void *ws, size_t ws_bytes, void *stream) {
  const int st = check_adapters(M, W, ad);
  if (st) return st;
  if (!rows_ok(X, M) || !rows_ok(Y, M) || !bf16_opt(T_out)) return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  const int64_t N = W->rows, K = W->cols;
  FwdParts f{};
  const size_t need = carve_fwd(ws, M, N, K, ad->count, ad->r, &f);
  if (!ws || !aligned(ws, 16) || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const AdapterSet set = set_of(ad);
  const NF4View w = view_of(W);
  uint16_t *T = T_out ? T_out : f.T;
  const int m = static_cast<int>(M);
  if (M <= kAdSmall) return from_hip(launch_ad_small(X, m, w, set, T, Y, f.sums, s));
  AdPrepare prep{};
  prep.index = set.index;
  prep.plan = f.plan;
  prep.w = w;
  prep.Wd = f.Wd;
  prep.M = m;
  prep.n = set.n;
  prep.r = set.r;
  hipError_t e = launch_ad_prepare(prep, s);
  if (e == hipSuccess) e = launch_ad_down(X, m, w.K, set.A, set, f.plan, f.part, T, s);
  if (e == hipSuccess) e = launch_ad_matmul_fwd(X, m, w.N, w.K, f.Wd, T, set.B, set.r, f.plan, f.tiles, Y, s);
  return from_hip(e);
}

int qlora_adapter_linear_bwd(const uint16_t *dY, const uint16_t *X, const uint16_t *T, int64_t M, const qlora_nf4_weight *W,
                             const qlora_adapters *ad, uint16_t *dX, uint16_t *dA, uint16_t *dB, void *ws, size_t ws_bytes,
                             void *stream) {
  const int st = check_adapters(M, W, ad);
  if (st) return st;
  if (!rows_ok(dY, M) || !rows_ok(X, M) || !bf16_opt(T) || !bf16_opt(dX) || !bf16_opt(dA) || !bf16_opt(dB))
    return QLORA_ERR_INVALID_ARG;
  if (M == 0 || (!dX && !dA && !dB)) return QLORA_OK;
  const int64_t N = W->rows, K = W->cols;
  BwdParts b{};
  const size_t need = carve_bwd(ws, M, N, K, ad->count, ad->r, &b);
  if (!ws || !aligned(ws, 16) || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const AdapterSet set = set_of(ad);
  const NF4View w = view_of(W);
  const int m = static_cast<int>(M), Np = static_cast<int>(round_up(N, 64));
  AdPrepare prep{};
  prep.index = set.index;
  prep.plan = b.plan;
  prep.w = w;
  prep.M = m;
  prep.n = set.n;
  prep.r = set.r;
  prep.Np = Np;
  const uint16_t *dYp = dY;
  if (dX || dA) {
    prep.B = set.B;
    prep.Bt = b.Bt;
    if (Np > N) {
      prep.dY = dY;
      prep.dYp = b.dYp;
      dYp = b.dYp;
    }
  }
  if (dX) {
    prep.A = set.A;
    prep.At = b.At;
    prep.Wd = b.Wd;
  }
  hipError_t e = launch_ad_prepare(prep, s);
  if (e == hipSuccess && dB && !T) {
    e = launch_ad_down(X, m, w.K, set.A, set, b.plan, b.part, b.T, s);
    T = b.T;
  }
  if (e == hipSuccess && (dX || dA)) e = launch_ad_down(dYp, m, Np, b.Bt, set, b.plan, b.part, b.G, s);
  if (e == hipSuccess && dX) e = launch_ad_matmul_dx(dYp, Np, m, w.N, w.K, b.Wd, b.G, b.At, set.r, b.plan, b.tiles, dX, s);
  if (e == hipSuccess && (dA || dB)) e = launch_ad_grads(X, dY, b.G, T, m, w.N, w.K, set, b.plan, dA, dB, s);
  return from_hip(e);
}

}  // extern "C"
