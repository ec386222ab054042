// Low-rank adapters beside a shared projection: the sequence of products behind lora_run and lora_backward
// (include/wqmlp_adapters.h).  Forward: t = scale x a^T, out = y + t b^T.  Backward: t = scale x a^T and
// dt = scale dy b, then db from t and dy, da from dt and x, dx = dx0 + dt a.
#include <algorithm>

#include "lora_common.h"

namespace wq {

namespace {

// Workspace: the terms of t, backward also those of dt, [3][M][R] bfloat16 each; then the parts of a split contraction, of
// either product in turn; then, backward, those of db's and of da's rows.  x's type is not known here: the float32 need covers it.
struct LoraWs {
  size_t dt, parts, db_parts, da_parts, total;
};
LoraWs lora_ws(int M, int K, int N, int E, int R, bool backward) {
  const size_t terms = align256((size_t)3 * M * R * 2);
  LoraWs w{};
  w.dt = terms;
  w.parts = terms * (backward ? 2 : 1);
  size_t p = std::max(lora_shrink_bytes(M, K, R, X_F32), lora_shrink_bytes(M, K, R, X_BF16));
  if (backward) p = std::max({p, lora_shrink_bytes(M, N, R, X_F32), lora_shrink_bytes(M, N, R, X_BF16)});
  w.db_parts = w.parts + align256(p);
  w.da_parts = w.db_parts + (backward ? align256(lora_outer_bytes(M, N, E, R)) : 0);
  w.total = w.da_parts + (backward ? align256(lora_outer_bytes(M, K, E, R)) : 0);
  return w;
}

}  // namespace

size_t lora_scratch_bytes(int M, int K, int N, int E, int R, bool backward) {
  return !backward && lora_one_launch(M, K, N, R) ? 0 : lora_ws(M, K, N, E, R, backward).total;
}

hipError_t launch_lora(int M, int K, int N, int E, int R, const void* x, XType xt, const void* a, const void* b, XType wt,
                       const float* scale, const int32_t* ids, const float* y, void* ws, float* out, hipStream_t st) {
  if (lora_one_launch(M, K, N, R)) return lora_rows(M, K, N, E, R, x, xt, a, b, wt, scale, ids, y, out, st);
  const LoraWs L = lora_ws(M, K, N, E, R, false);
  uint8_t* p = reinterpret_cast<uint8_t*>(ws);
  uint16_t* t = reinterpret_cast<uint16_t*>(p);
  const bool few = lora_few_rows(M, K, N, R, wt);
  hipError_t err = lora_shrink(few, M, K, E, R, x, xt, a, wt, false, scale, ids, t, reinterpret_cast<float*>(p + L.parts), st);
  if (err == hipSuccess) err = lora_expand(few, M, N, E, R, t, b, wt, false, ids, y, out, X_F32, st);
  return err;
}

hipError_t launch_lora_backward(int M, int K, int N, int E, int R, const void* dy, XType dyt, const void* x, XType xt,
                                const void* a, const void* b, XType wt, const float* scale, const int32_t* ids,
                                const void* dx0, XType dxt, void* ws, void* dx, float* da, float* db, hipStream_t st) {
  const LoraWs L = lora_ws(M, K, N, E, R, true);
  uint8_t* p = reinterpret_cast<uint8_t*>(ws);
  uint16_t* t = reinterpret_cast<uint16_t*>(p);
  uint16_t* dt = reinterpret_cast<uint16_t*>(p + L.dt);
  float* parts = reinterpret_cast<float*>(p + L.parts);
  const bool few = lora_few_rows(M, K, N, R, wt);
  // Each pass over dy (or x) follows the other one directly, so that it finds a part of it in the last-level cache (4096 x 17408
  // float32: 47 us instead of 57); da and db in one launch, for operands of one type, come after both products instead.
  const bool together = da != nullptr && db != nullptr && xt == dyt;
  const OuterJob jobs[2] = {{N, t, dy, dyt, true, db, reinterpret_cast<float*>(p + L.db_parts)},
                            {K, dt, x, xt, false, da, reinterpret_cast<float*>(p + L.da_parts)}};
  hipError_t err = hipSuccess;
  if (db != nullptr) {
    if (M > 0) err = lora_shrink(few, M, K, E, R, x, xt, a, wt, false, scale, ids, t, parts, st);
    if (err == hipSuccess && !together) err = lora_outer(M, E, R, jobs, 1, ids, st);
  }
  if (err == hipSuccess && (da != nullptr || dx != nullptr) && M > 0)
    err = lora_shrink(few, M, N, E, R, dy, dyt, b, wt, true, scale, ids, dt, parts, st);
  if (err == hipSuccess && together) err = lora_outer(M, E, R, jobs, 2, ids, st);
  else if (err == hipSuccess && da != nullptr) err = lora_outer(M, E, R, jobs + 1, 1, ids, st);
  if (err == hipSuccess && (da != nullptr || db != nullptr))
    err = lora_outer_join(M, E, R, db != nullptr ? jobs : jobs + 1, (db != nullptr) + (da != nullptr), st);
  if (err == hipSuccess && dx != nullptr && M > 0) err = lora_expand(few, M, K, E, R, dt, a, wt, true, ids, dx0, dx, dxt, st);
  return err;
}

}  // namespace wq
