// Low-rank adapters beside a shared projection: the sequence of products behind lora_run and lora_backward
// (include/wqmlp_adapters.h).  Forward: t = x a^T, out = y + scale t b^T.  Backward: t = x a^T and dt = dy b, then
// db from t and dy, da from dt and x, dx = dx0 + scale dt a.  t and dt are float32 in the workspace, in the parts
// that the split contraction left; whoever reads them adds the parts in order and multiplies by scale.
#include <algorithm>

#include "lora_common.h"

namespace wq {

namespace {

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Workspace: t parts [S][M][R]; backward also dt parts and the larger of the weight gradients' row parts.
struct LoraWs {
  int s, sd;
  size_t dt, parts, total;
};
LoraWs lora_ws(int M, int K, int N, int E, int R, bool backward) {
  LoraWs w{};
  w.s = lora_shrink_parts(M, K, R);
  w.total = w.dt = up256((size_t)w.s * M * R * 4);
  if (backward) {
    w.sd = lora_shrink_parts(M, N, R);
    w.parts = w.dt + up256((size_t)w.sd * M * R * 4);
    w.total = w.parts + up256(std::max(lora_outer_bytes(M, K, E, R), lora_outer_bytes(M, N, E, R)));
  }
  return w;
}

}  // namespace

size_t lora_scratch_bytes(int M, int K, int N, int E, int R, bool backward) {
  return lora_ws(M, K, N, E, R, backward).total;
}

hipError_t launch_lora(int M, int K, int N, int E, int R, const void* x, XType xt, const void* a, const void* b, XType wt,
                       const float* scale, const int32_t* ids, const float* y, void* ws, float* out, hipStream_t st) {
  const LoraWs L = lora_ws(M, K, N, E, R, false);
  float* t = reinterpret_cast<float*>(ws);
  hipError_t err = lora_shrink(M, K, E, R, L.s, x, xt, a, wt, false, ids, t, st);
  if (err == hipSuccess) err = lora_expand(M, N, E, R, L.s, t, b, wt, false, scale, ids, y, out, X_F32, st);
  return err;
}

hipError_t launch_lora_backward(int M, int K, int N, int E, int R, const void* dy, XType dyt, const void* x, XType xt,
                                const void* a, const void* b, XType wt, const float* scale, const int32_t* ids,
                                const void* dx0, XType dxt, void* ws, void* dx, float* da, float* db, hipStream_t st) {
  const LoraWs L = lora_ws(M, K, N, E, R, true);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  float* t = reinterpret_cast<float*>(base);
  float* dt = reinterpret_cast<float*>(base + L.dt);
  float* parts = reinterpret_cast<float*>(base + L.parts);
  hipError_t err = hipSuccess;
  if (db != nullptr) {
    if (M > 0) err = lora_shrink(M, K, E, R, L.s, x, xt, a, wt, false, ids, t, st);
    if (err == hipSuccess) err = lora_outer(M, N, E, R, L.s, t, dy, dyt, true, scale, ids, db, parts, st);
  }
  if (da == nullptr && dx == nullptr) return err;
  if (err == hipSuccess && M > 0) err = lora_shrink(M, N, E, R, L.sd, dy, dyt, b, wt, true, ids, dt, st);
  if (err == hipSuccess && da != nullptr) err = lora_outer(M, K, E, R, L.sd, dt, x, xt, false, scale, ids, da, parts, st);
  if (err == hipSuccess && dx != nullptr && M > 0)
    err = lora_expand(M, K, E, R, L.sd, dt, a, wt, true, scale, ids, dx0, dx, dxt, st);
  return err;
}

}  // namespace wq
