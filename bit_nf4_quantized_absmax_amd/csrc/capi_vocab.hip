// C ABI of the losses over the vocabulary: argument validation and launches.
// Every check runs before anything is launched.
#include <math.h>

#include "capi_util.h"

using namespace qlora;

namespace {

int elem_bytes(int32_t type) { return type == 0 ? 4 : 2; }

// A kernel's offsets within a row: bytes in 32 bits, words in 31, up to a
// gradient workgroup's part (less than 2^23 bytes) past its end.
constexpr int64_t kMaxRowBytes = (int64_t{1} << 32) - (int64_t{1} << 24);

int check_rows(int32_t type, int64_t M, int64_t V) {
  if (type < 0 || type > QLORA_IN_FP16 || M < 0 || V < 1) return QLORA_ERR_INVALID_ARG;
  if (V > kMaxRowBytes / elem_bytes(type) || M > kMaxThreads) return QLORA_ERR_UNSUPPORTED_SHAPE;
  return QLORA_OK;
}

// Whether the launch of M rows of so many threads can be counted.
bool launch_ok(int64_t M, int64_t row_threads) { return M <= kMaxThreads / row_threads; }

bool sums_ok(int32_t type, int64_t M, int64_t V, int32_t top) { return M == 0 || launch_ok(M, vocab_row_threads(M, V, type, top)); }

bool distill_bwd_ok(int32_t type, int64_t M, int64_t V) { return M == 0 || launch_ok(M, distill_bwd_row_threads(M, V, type)); }

// Logits (or their gradient): pitch, presence and the element's alignment.
int check_matrix(const void *p, int32_t type, int64_t M, int64_t V, int64_t ld) {
  if (ld < V) return QLORA_ERR_INVALID_ARG;
  if ((M > 0 && !p) || !aligned(p, elem_bytes(type))) return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

bool present(const void *p, int64_t M, uintptr_t a) { return (M == 0 || p) && aligned(p, a); }

int check_logits(const qlora_logits *l) {
  if (!l) return QLORA_ERR_INVALID_ARG;
  const int st = check_rows(l->type, l->rows, l->words);
  return st ? st : check_matrix(l->z, l->type, l->rows, l->words, l->pitch);
}

int check_teacher(const qlora_teacher *t, int64_t M) {
  if (!t) return QLORA_ERR_INVALID_ARG;
  if (t->count < 1 || t->count > kDistillMax) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (!present(t->index, M, 8) || !present(t->logit, M, 4)) return QLORA_ERR_INVALID_ARG;
  if (!isfinite(t->temperature) || !(t->temperature > 0.f)) return QLORA_ERR_INVALID_ARG;
  const float c = 1.442695f / t->temperature;
  if (!isfinite(c) || c == 0.f) return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

Logits view_of(const qlora_logits *l) { return Logits{l->z, l->type, l->rows, l->words, l->pitch}; }
Teacher view_of(const qlora_teacher *t) { return Teacher{t->index, t->logit, t->count, t->temperature}; }

bool ws_ok(const void *ws, size_t have, size_t need) { return need == 0 || (ws && aligned(ws, 16) && have >= need); }

}  // namespace

extern "C" {

size_t qlora_vocab_workspace_bytes(int32_t type, int64_t rows, int64_t words, int32_t top) {
  if (check_rows(type, rows, words) || rows == 0 || top < 0 || top > kTopMax || top > words) return 0;
  if (!sums_ok(type, rows, words, top)) return 0;
  return vocab_ws_bytes(rows, words, type, top);
}

int qlora_token_logprobs(const qlora_logits *l, const int64_t *target, int32_t top, float *logprob, float *entropy,
                         float *lse, float *top_logprob, int64_t *top_index, void *ws, size_t ws_bytes, void *stream) {
  const int st = check_logits(l);
  if (st) return st;
  const int64_t M = l->rows;
  if (top < 0 || top > kTopMax || top > l->words || !sums_ok(l->type, M, l->words, top)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (!present(target, M, 8) || !present(logprob, M, 4) || !present(entropy, M, 4) || !present(lse, M, 4))
    return QLORA_ERR_INVALID_ARG;
  if (top > 0 && (!present(top_logprob, M, 4) || !present(top_index, M, 8))) return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  if (!ws_ok(ws, ws_bytes, vocab_ws_bytes(M, l->words, l->type, top))) return QLORA_ERR_WORKSPACE;
  return from_hip(launch_token_logprobs(view_of(l), target, top, logprob, entropy, lse, top_logprob, top_index, ws,
                                        static_cast<hipStream_t>(stream)));
}

int qlora_token_logprobs_bwd(const qlora_logits *l, const int64_t *target, const float *lse, const float *entropy,
                             const float *g_logprob, const float *g_entropy, void *dz, int64_t dz_pitch, void *stream) {
  int st = check_logits(l);
  if (!st) st = check_matrix(dz, l->type, l->rows, l->words, dz_pitch);
  if (st) return st;
  const int64_t M = l->rows;
  if (!launch_ok(M, logprobs_bwd_row_threads(l->words, l->type))) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (!present(target, M, 8) || !present(lse, M, 4) || !present(entropy, M, 4) || !aligned(g_logprob, 4) ||
      !aligned(g_entropy, 4))
    return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  return from_hip(launch_token_logprobs_bwd(view_of(l), target, lse, entropy, g_logprob, g_entropy, dz, dz_pitch,
                                            static_cast<hipStream_t>(stream)));
}

int qlora_distill_fwd(const qlora_logits *l, const qlora_teacher *t, float *loss, float *lse, void *ws, size_t ws_bytes,
                      void *stream) {
  int st = check_logits(l);
  if (!st) st = check_teacher(t, l->rows);
  if (st) return st;
  const int64_t M = l->rows;
  if (!sums_ok(l->type, M, l->words, 0)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (!present(loss, M, 4) || !present(lse, M, 4)) return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  if (!ws_ok(ws, ws_bytes, vocab_ws_bytes(M, l->words, l->type, 0))) return QLORA_ERR_WORKSPACE;
  return from_hip(launch_distill_fwd(view_of(l), view_of(t), loss, lse, ws, static_cast<hipStream_t>(stream)));
}

int qlora_distill_bwd(const qlora_logits *l, const qlora_teacher *t, const float *lse, const float *weight, void *dz,
                      int64_t dz_pitch, void *stream) {
  int st = check_logits(l);
  if (!st) st = check_teacher(t, l->rows);
  if (!st) st = check_matrix(dz, l->type, l->rows, l->words, dz_pitch);
  if (st) return st;
  if (!distill_bwd_ok(l->type, l->rows, l->words)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (!present(lse, l->rows, 4) || !aligned(weight, 4)) return QLORA_ERR_INVALID_ARG;
  if (l->rows == 0) return QLORA_OK;
  return from_hip(
      launch_distill_bwd(view_of(l), view_of(t), lse, weight, dz, dz_pitch, static_cast<hipStream_t>(stream)));
}

int qlora_distill(const qlora_logits *l, const qlora_teacher *t, const float *weight, float *loss, float *lse, void *dz,
                  int64_t dz_pitch, void *ws, size_t ws_bytes, void *stream) {
  int st = check_logits(l);
  if (!st) st = check_teacher(t, l->rows);
  if (!st) st = check_matrix(dz, l->type, l->rows, l->words, dz_pitch);
  if (st) return st;
  const int64_t M = l->rows;
  if (!sums_ok(l->type, M, l->words, 0) || !distill_bwd_ok(l->type, M, l->words)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (!present(loss, M, 4) || !present(lse, M, 4) || !aligned(weight, 4)) return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  if (!ws_ok(ws, ws_bytes, vocab_ws_bytes(M, l->words, l->type, 0))) return QLORA_ERR_WORKSPACE;
  return from_hip(launch_distill(view_of(l), view_of(t), weight, loss, lse, dz, dz_pitch, ws,
                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
