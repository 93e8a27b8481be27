// C ABI of the cross entropy through the output head: argument validation, the cut
// of the vocabulary, workspace carving and the passes.  Every check runs before
// anything is launched.
#include <algorithm>

#include "capi_util.h"

using namespace qlora;

namespace {

constexpr int64_t kMaxRows = int64_t{1} << 22;
constexpr int64_t kMaxK = int64_t{1} << 18;

int check_shape(int64_t M, int64_t V, int64_t K) {
  if (M < 0 || V < 1 || K < 1) return QLORA_ERR_INVALID_ARG;
  if (K % 64 != 0 || K > kMaxK || V > kMaxElems || M > kMaxRows || M > kMaxElems / K) return QLORA_ERR_UNSUPPORTED_SHAPE;
  return QLORA_OK;
}

// Words of a piece: as many as keep `budget` values of it, a multiple of 256 (one
// tile) at least, and K times them within 32-bit offsets.
int64_t piece_words(int64_t M, int64_t V, int64_t K, int64_t budget) {
  int64_t w = std::max<int64_t>(256, budget / M / 256 * 256);
  w = std::min(w, std::max<int64_t>(256, (int64_t{1} << 30) / K / 256 * 256));
  return std::min<int64_t>(w, round_up(V, 64));
}

// E of a piece: 2^27 values of 2 bytes, as the memory-side cache has (8192 x 32000 x 4096,
// loss and dX: 2895 us with 2^26, whose pieces have more launches' ends and additions to
// the gradient, 2735 with 2^27, 2716 with 2^28, which is not worth its memory).
// Without a gradient only the group sums are kept, 8 bytes for 64 words.
constexpr int64_t kPieceE = int64_t{1} << 27, kPieceSums = int64_t{1} << 28;

struct Parts {
  HeadRows h;
  HeadPiece pc;
  uint16_t *Xc;
  float *C;
  uint16_t *Zt;
  int64_t words;
  HeadCut cut;
};

size_t carve(void *ws, int64_t M, int64_t V, int64_t K, int32_t pass, Parts *p) {
  Carve c(ws);
  p->h.place = c.take<int>(M);
  p->h.list = c.take<int>(M);
  p->h.tgt = c.take<int>(M);
  p->h.count = c.take<int>(1);
  if (pass == QLORA_HEAD_DW) {
    const int64_t depth = head_dw_depth(M);
    p->Xc = c.take<uint16_t>(depth * K);
    p->words = piece_words(depth, V, K, kPieceE);
    p->Zt = c.take<uint16_t>(p->words * depth);
    return c.used;
  }
  p->h.zt = c.take<float>(M);
  p->h.ref = c.take<float>(M);
  p->h.sum = c.take<double>(M);
  p->h.factor = c.take<float>(M);
  p->words = piece_words(M, V, K, pass == QLORA_HEAD_DX ? kPieceE : kPieceSums);
  p->pc.rows = static_cast<int>(M);
  p->pc.part = c.take<float2>((p->words + 63) / 64 * M);
  if (pass == QLORA_HEAD_DX) {
    p->cut = head_cut(M, K, p->words);
    p->pc.E = c.take<uint16_t>(p->words * M);
    p->C = c.take<float>(static_cast<size_t>(p->cut.most) * M * K);
  }
  return c.used;
}

bool rows8(const void *p, int64_t M, uintptr_t a) { return (M == 0 || p) && aligned(p, a); }

}  // namespace

extern "C" {

size_t qlora_head_workspace_bytes(int64_t M, int64_t V, int64_t K, int32_t pass) {
  if (check_shape(M, V, K) || M == 0 || pass < QLORA_HEAD_LOSS || pass > QLORA_HEAD_DW) return 0;
  Parts p{};
  return carve(nullptr, M, V, K, pass, &p);
}

int qlora_head_cross_entropy(const uint16_t *X, int64_t M, const uint16_t *W, int64_t V, int64_t K, const int64_t *target,
                             const float *weight, float *loss, float *lse, void *dX, int32_t dx_fp32, void *ws, size_t ws_bytes,
                             void *stream) {
  const int st = check_shape(M, V, K);
  if (st) return st;
  if (!rows_ok(X, M) || !bf16_ok(W) || !rows8(target, M, 8) || !aligned(weight, 4) || !rows8(loss, M, 4) || !rows8(lse, M, 4) ||
      !aligned(dX, 16) || dx_fp32 < 0 || dx_fp32 > 1)
    return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  Parts p{};
  const size_t need = carve(ws, M, V, K, dX ? QLORA_HEAD_DX : QLORA_HEAD_LOSS, &p);
  if (!ws || !aligned(ws, 16) || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int m = static_cast<int>(M), k = static_cast<int>(K), v = static_cast<int>(V);
  const bool small = M <= kHeadSmall, at_once = small && !dX && p.words >= V;
  hipError_t e = hipSuccess;
  if (!small) e = launch_head_rows(target, m, v, p.h, s);
  for (int64_t v0 = 0; v0 < V && e == hipSuccess; v0 += p.words) {
    const int words = static_cast<int>(std::min<int64_t>(p.words, V - v0));
    p.pc.pitch = static_cast<int>(round_up(words, 64));
    if (small)
      e = launch_head_small_piece(X, target, m, W, v, k, static_cast<int>(v0), words, v0 == 0, p.h, p.pc, p.cut, dX ? p.C : nullptr,
                                  at_once ? loss : nullptr, at_once ? lse : nullptr, s);
    else
      e = launch_head_piece(X, m, W, v, k, static_cast<int>(v0), words, v0 == 0, p.h, p.pc, p.cut, dX ? p.C : nullptr, s);
  }
  if (e == hipSuccess && !at_once) e = launch_head_finish(W, M, k, weight, p.h, p.cut, p.C, loss, lse, dX, dX ? 1 + dx_fp32 : 0, s);
  return from_hip(e);
}

int qlora_head_scale(const float *D, int64_t M, int64_t V, int64_t K, const int64_t *target, const float *g, uint16_t *dX, void *stream) {
  const int st = check_shape(M, V, K);
  if (st) return st;
  if (!rows8(D, M, 16) || !rows8(target, M, 8) || !rows8(g, M, 4) || !rows_ok(dX, M)) return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  return from_hip(launch_head_scale(D, M, static_cast<int>(K), target, static_cast<int>(V), g, dX, static_cast<hipStream_t>(stream)));
}

int qlora_head_cross_entropy_dW(const uint16_t *X, int64_t M, const uint16_t *W, int64_t V, int64_t K, const int64_t *target,
                                const float *lse, const float *weight, uint16_t *dW, void *ws, size_t ws_bytes, void *stream) {
  const int st = check_shape(M, V, K);
  if (st) return st;
  if (!rows_ok(X, M) || !bf16_ok(W) || !rows8(target, M, 8) || !rows8(lse, M, 4) || !aligned(weight, 4) || !bf16_ok(dW))
    return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  Parts p{};
  const size_t need = carve(ws, M, V, K, QLORA_HEAD_DW, &p);
  if (!ws || !aligned(ws, 16) || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int m = static_cast<int>(M), k = static_cast<int>(K);
  hipError_t e = launch_head_rows(target, m, static_cast<int>(V), p.h, s);
  if (e == hipSuccess) e = launch_head_gather(X, m, k, p.h, p.Xc, s);
  for (int64_t v0 = 0; v0 < V && e == hipSuccess; v0 += p.words)
    e = launch_head_dw(p.Xc, m, W, k, static_cast<int>(v0), static_cast<int>(std::min<int64_t>(p.words, V - v0)), p.h, lse, weight, p.Zt,
                       dW, s);
  return from_hip(e);
}

}  // extern "C"
