// C ABI of the gradient norm: argument validation, the cut into chunks and the
// launches.  Every check runs before anything is launched.
#include <algorithm>

#include "capi_util.h"

using namespace qlora;

namespace {

constexpr int kMaxTensors = 1 << 16;
constexpr int kMaxGroups = 1 << 12;
constexpr int64_t kMinChunk = 4096;         // elements: 16 a thread
constexpr int64_t kChunks = 2048;           // 8 workgroups a compute unit
constexpr int64_t kMaxChunks = int64_t{1} << 23;

struct Plan {
  int64_t chunk = kMinChunk, stride = 0;
};

// The cut: about kChunks chunks in all, whole multiples of kMinChunk; every part of
// a tensor has chunks of its own.
int make_plan(int32_t count, const qlora_grad_tensor *t, int32_t groups, Plan *p) {
  if (count < 0 || (count > 0 && !t) || groups < 1) return QLORA_ERR_INVALID_ARG;
  if (count > kMaxTensors || groups > kMaxGroups) return QLORA_ERR_UNSUPPORTED_SHAPE;
  int64_t all = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].count < 0 || t[i].type < 0 || t[i].type > QLORA_IN_FP16) return QLORA_ERR_INVALID_ARG;
    if (t[i].count % groups != 0 || t[i].count > (int64_t{1} << 40)) return QLORA_ERR_UNSUPPORTED_SHAPE;
    all += t[i].count;
  }
  p->chunk = std::max(kMinChunk, (all / kChunks + kMinChunk - 1) / kMinChunk * kMinChunk);
  if (p->chunk > kMaxElems / 2) return QLORA_ERR_UNSUPPORTED_SHAPE;
  for (int32_t i = 0; i < count; ++i) p->stride += (t[i].count / groups + p->chunk - 1) / p->chunk;
  return p->stride * groups > kMaxChunks ? QLORA_ERR_UNSUPPORTED_SHAPE : QLORA_OK;
}

GradPlan carve(void *ws, const Plan &p, int32_t groups, size_t *bytes) {
  Carve c(ws);
  GradPlan g;
  g.table = c.take<GradChunk>(p.stride * groups);
  g.sums = c.take<double>(p.stride * groups);
  g.groups = groups;
  g.stride = static_cast<int>(p.stride);
  g.chunk = static_cast<int>(p.chunk);
  *bytes = c.used;
  return g;
}

int run(int32_t count, const qlora_grad_tensor *t, int32_t groups, const float *max_norm, float *norm, void *ws, size_t ws_bytes,
        void *stream) {
  Plan plan;
  const int st = make_plan(count, t, groups, &plan);
  if (st) return st;
  if (!norm || !aligned(norm, 4) || (max_norm && !(*max_norm >= 0.f))) return QLORA_ERR_INVALID_ARG;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].count == 0) continue;
    const uintptr_t width = t[i].type == 0 ? 4 : 2;
    if (!t[i].x || !aligned(t[i].x, width) || (max_norm && (!t[i].out || !aligned(t[i].out, width)))) return QLORA_ERR_INVALID_ARG;
  }
  size_t need = 0;
  const GradPlan g = carve(ws, plan, groups, &need);
  if (need > 0 && (!ws || !aligned(ws, 16) || ws_bytes < need)) return QLORA_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  GradList list;
  list.n = 0;
  int64_t first = 0;
  bool lead = true;
  hipError_t e = hipSuccess;
  for (int32_t i = 0; i < count && e == hipSuccess; ++i) {
    if (t[i].count > 0) {
      const int64_t part = t[i].count / groups;
      list.t[list.n++] = GradTensor{t[i].x, max_norm ? t[i].out : nullptr, part, static_cast<int>(t[i].type), static_cast<int>(first)};
      first += (part + plan.chunk - 1) / plan.chunk;
    }
    if (list.n > 0 && (list.n == kGradList || i + 1 == count)) {
      list.chunks = static_cast<int>(first) - list.t[0].first;
      e = launch_grad_squares(list, g, lead, s);
      lead = false;
      list.n = 0;
    }
  }
  if (e == hipSuccess) e = launch_grad_norm(g, max_norm, norm, s);
  return from_hip(e);
}

}  // namespace

extern "C" {

size_t qlora_grad_norm_workspace_bytes(int32_t count, const qlora_grad_tensor *t, int32_t groups) {
  Plan plan;
  if (make_plan(count, t, groups, &plan)) return 0;
  size_t need = 0;
  carve(nullptr, plan, groups, &need);
  return need;
}

int qlora_grad_norm(int32_t count, const qlora_grad_tensor *t, int32_t groups, float *norm, void *ws, size_t ws_bytes, void *stream) {
  return run(count, t, groups, nullptr, norm, ws, ws_bytes, stream);
}

int qlora_clip_grad_norm(int32_t count, const qlora_grad_tensor *t, int32_t groups, float max_norm, float *norm, void *ws, size_t ws_bytes,
                         void *stream) {
  return run(count, t, groups, &max_norm, norm, ws, ws_bytes, stream);
}

}  // extern "C"
