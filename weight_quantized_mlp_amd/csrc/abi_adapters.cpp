// C ABI of the adapter, input-gradient and AdamW calls (declarations and contracts: include/wqmlp_adapters.h).
// The checks come in the two phases of abi.cpp: arithmetic on the arguments, then the device.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <utility>
#include <vector>

#include "../../include/wqmlp_adapters.h"
#include "abi_common.h"
#include "launch.h"

namespace {

using namespace wq::abi;

static_assert(wq::kAdamwKeepV == WQ_ADAMW_KEEP_V, "one flag");

bool is_float(int dt) { return dt == WQ_F32 || dt == WQ_BF16 || dt == WQ_F16; }
wq::XType xtype(int dt) { return dt == WQ_F32 ? wq::X_F32 : (dt == WQ_BF16 ? wq::X_BF16 : wq::X_F16); }

bool lora_shape_ok(int64_t M, int64_t K, int64_t N, int64_t E, int64_t R) {
  if (M < 0 || M > kMaxDim || K <= 0 || K > kMaxDim || K % 16 || N <= 0 || N > kMaxDim) return false;
  if (E <= 0 || E > kMaxDim || R < 8 || R > WQ_LORA_MAX_RANK || R % 8) return false;
  return M * std::max(K, N) <= kMaxElems && E * R <= kMaxElems / std::max(K, N);
}

bool grad_shape_ok(int fmt, int64_t M, int64_t N, int64_t K) {
  if (fmt != WQ_FMT_FP8W && fmt != WQ_FMT_NVFP4) return false;
  if (M < 0 || M > kMaxDim || N <= 0 || N > kMaxDim || K <= 0 || K > kMaxDim) return false;
  if (K % (fmt == WQ_FMT_NVFP4 ? 64 : 16)) return false;
  return M * std::max(N, K) <= kMaxElems;
}

}  // namespace

extern "C" {

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t E, int64_t R, int backward) {
  if (!lora_shape_ok(M, K, N, E, R) || (backward != 0 && backward != 1)) return 0;
  return wq::lora_scratch_bytes((int)M, (int)K, (int)N, (int)E, (int)R, backward != 0);
}

int lora_run(int64_t M, int64_t K, int64_t N, int64_t E, int64_t R, const void* x, int x_dtype, const void* a,
             const void* b, int w_dtype, const float* scale, const int32_t* ids, const float* y, void* workspace,
             size_t workspace_bytes, float* out, void* stream) {
  if (!is_float(x_dtype) || !is_float(w_dtype) || !lora_shape_ok(M, K, N, E, R)) return WQ_EINVAL;
  if (any_null({a, b, scale})) return WQ_EINVAL;
  if (M == 0) return WQ_OK;
  if (any_null({x, ids, out})) return WQ_EINVAL;
  if (!all_aligned({x, a, b, scale, ids, y, workspace, out})) return WQ_EALIGN;
  const size_t need = lora_workspace_bytes(M, K, N, E, R, 0);
  if (need && (workspace == nullptr || workspace_bytes < need)) return WQ_EWORKSPACE;
  const Rng ry{y, y == nullptr || y == out ? 0 : (size_t)M * N * 4};   // in place, or apart
  if (any_overlap({{out, (size_t)M * N * 4}, {workspace, need}},
                  {{x, (size_t)M * K * xsize(x_dtype)}, {a, (size_t)E * R * K * xsize(w_dtype)},
                   {b, (size_t)E * N * R * xsize(w_dtype)}, {scale, (size_t)E * 4}, {ids, (size_t)M * 4}, ry}))
    return WQ_EOVERLAP;
  const int rc = check_device({x, a, b, scale, ids, y, need ? workspace : nullptr, out});
  if (rc != WQ_OK) return rc;
  return launched(wq::launch_lora((int)M, (int)K, (int)N, (int)E, (int)R, x, xtype(x_dtype), a, b, xtype(w_dtype), scale,
                                  ids, y, workspace, out, reinterpret_cast<hipStream_t>(stream)));
}

int lora_backward(int64_t M, int64_t K, int64_t N, int64_t E, int64_t R, const void* dy, int dy_dtype, const void* x,
                  int x_dtype, const void* a, const void* b, int w_dtype, const float* scale, const int32_t* ids,
                  const void* dx0, int dx_dtype, void* workspace, size_t workspace_bytes, void* dx, float* da, float* db,
                  void* stream) {
  if ((dy_dtype != WQ_F32 && dy_dtype != WQ_BF16) || !is_float(x_dtype) || !is_float(w_dtype) || !is_float(dx_dtype))
    return WQ_EINVAL;
  if (!lora_shape_ok(M, K, N, E, R)) return WQ_EINVAL;
  if (any_null({a, b, scale})) return WQ_EINVAL;
  if (M > 0 && dx == nullptr && da == nullptr && db == nullptr) return WQ_EINVAL;
  if (M == 0) {   // no rows: dx is empty (and may be NULL, as an empty tensor's address is), the weight gradients are zero
    dx = nullptr;
    if (da == nullptr && db == nullptr) return WQ_OK;
    dy = x = dx0 = nullptr;
    ids = nullptr;
  } else if (any_null({dy, x, ids})) {
    return WQ_EINVAL;
  }
  if (dx == nullptr) dx0 = nullptr;
  if (!all_aligned({dy, x, a, b, scale, ids, dx0, workspace, dx, da, db})) return WQ_EALIGN;
  const size_t need = lora_workspace_bytes(M, K, N, E, R, 1);
  if (need && (workspace == nullptr || workspace_bytes < need)) return WQ_EWORKSPACE;
  const size_t nx = dx ? (size_t)M * K * xsize(dx_dtype) : 0;
  if (any_overlap({{dx, nx}, {da, da ? (size_t)E * R * K * 4 : 0}, {db, db ? (size_t)E * N * R * 4 : 0}, {workspace, need}},
                  {{dy, (size_t)M * N * xsize(dy_dtype)}, {x, (size_t)M * K * xsize(x_dtype)},
                   {a, (size_t)E * R * K * xsize(w_dtype)}, {b, (size_t)E * N * R * xsize(w_dtype)},
                   {scale, (size_t)E * 4}, {ids, (size_t)M * 4}, {dx0, dx0 == nullptr || dx0 == dx ? 0 : nx}}))
    return WQ_EOVERLAP;
  const int rc = check_device({dy, x, a, b, scale, ids, dx0, need ? workspace : nullptr, dx, da, db});
  if (rc != WQ_OK) return rc;
  return launched(wq::launch_lora_backward((int)M, (int)K, (int)N, (int)E, (int)R, dy, xtype(dy_dtype), x, xtype(x_dtype),
                                           a, b, xtype(w_dtype), scale, ids, dx0, xtype(dx_dtype), workspace, dx, da, db,
                                           reinterpret_cast<hipStream_t>(stream)));
}

size_t qlinear_backward_workspace_bytes(int fmt, int64_t M, int64_t N, int64_t K, int dx_dtype) {
  if (!grad_shape_ok(fmt, M, N, K) || M == 0 || (dx_dtype != WQ_F32 && dx_dtype != WQ_BF16)) return 0;
  return wq::linear_grad_scratch_bytes(fmt == WQ_FMT_NVFP4 ? 1 : 0, (int)M, (int)N, (int)K, xtype(dx_dtype));
}

int qlinear_backward(int fmt, int64_t M, int64_t N, int64_t K, const void* dy, int dy_dtype, const uint8_t* w,
                     const float* scale, float global_scale, void* workspace, size_t workspace_bytes, void* dx,
                     int dx_dtype, void* stream) {
  if (!grad_shape_ok(fmt, M, N, K)) return WQ_EINVAL;
  if ((dy_dtype != WQ_F32 && dy_dtype != WQ_BF16) || (dx_dtype != WQ_F32 && dx_dtype != WQ_BF16)) return WQ_EINVAL;
  if (w == nullptr || (fmt == WQ_FMT_FP8W && scale == nullptr)) return WQ_EINVAL;
  if (fmt == WQ_FMT_NVFP4 && (!(global_scale > 0.f) || !std::isfinite(global_scale))) return WQ_EINVAL;
  if (M == 0) return WQ_OK;
  if (any_null({dy, dx})) return WQ_EINVAL;
  if (fmt == WQ_FMT_NVFP4) scale = nullptr;
  if (!all_aligned({dy, w, scale, workspace, dx})) return WQ_EALIGN;
  const size_t need = qlinear_backward_workspace_bytes(fmt, M, N, K, dx_dtype);
  if (need && (workspace == nullptr || workspace_bytes < need)) return WQ_EWORKSPACE;
  if (any_overlap({{dx, (size_t)M * K * xsize(dx_dtype)}, {workspace, need}},
                  {{dy, (size_t)M * N * xsize(dy_dtype)}, {w, wbytes(fmt, N, K)}, {scale, scale ? (size_t)N * 4 : 0}}))
    return WQ_EOVERLAP;
  const int rc = check_device({dy, w, scale, need ? workspace : nullptr, dx});
  if (rc != WQ_OK) return rc;
  return launched(wq::launch_linear_grad(fmt == WQ_FMT_NVFP4 ? 1 : 0, (int)M, (int)N, (int)K, dy, xtype(dy_dtype), w, scale,
                                         fmt == WQ_FMT_NVFP4 ? 1.0f / global_scale : 0.f, workspace, dx, xtype(dx_dtype),
                                         reinterpret_cast<hipStream_t>(stream)));
}

size_t adamw_table_bytes(int64_t count) {
  if (count <= 0 || count > WQ_ADAMW_MAX_TENSORS) return 0;
  return align256((size_t)wq::adamw_layout_bytes(count));
}

int adamw_table_build(int64_t count, const wq_adamw_tensor* tensors, int state_bits, void* table, size_t table_bytes,
                      void* stream) try {
  const bool b8 = state_bits == 8 || state_bits == (8 | WQ_ADAMW_KEEP_V);
  if (count <= 0 || count > WQ_ADAMW_MAX_TENSORS || (!b8 && state_bits != 32)) return WQ_EINVAL;
  if (tensors == nullptr || table == nullptr) return WQ_EINVAL;
  const size_t need = adamw_table_bytes(count);
  if (!all_aligned({table})) return WQ_EALIGN;
  if (table_bytes < need) return WQ_EWORKSPACE;
  struct Span {
    uintptr_t p, end;
    bool out;
  };
  std::vector<Span> spans;                 // what a step reads and writes, for one overlap check over all tensors
  std::vector<wq::AdamwEntry> entries((size_t)count);
  spans.reserve((size_t)count * 7 + 1);
  spans.push_back({(uintptr_t)table, (uintptr_t)table + need, true});   // written here, read by the steps
  int64_t chunks = 0, elems = 0;
  for (int64_t i = 0; i < count; ++i) {
    const wq_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > kMaxElems || (t.g_dtype != WQ_F32 && t.g_dtype != WQ_BF16)) return WQ_EINVAL;
    if (t.copy != nullptr && t.copy_dtype != WQ_BF16 && t.copy_dtype != WQ_F16) return WQ_EINVAL;
    elems += t.n;
    if (elems > kMaxElems) return WQ_EINVAL;
    entries[i] = {t.n, chunks, t.p, t.g, t.m, t.v, b8 ? t.m_scale : nullptr, b8 ? t.v_scale : nullptr, t.copy,
                  t.g_dtype, t.copy_dtype};
    chunks += wq::adamw_chunks(t.n);
    if (t.n == 0) continue;
    if (any_null({t.p, t.g, t.m, t.v}) || (b8 && any_null({t.m_scale, t.v_scale}))) return WQ_EINVAL;
    if (!all_aligned({t.p, t.g, t.m, t.v, entries[i].m_scale, entries[i].v_scale, t.copy})) return WQ_EALIGN;
    const size_t n = (size_t)t.n, ns = (n + WQ_ADAMW_BLOCK - 1) / WQ_ADAMW_BLOCK * 4, st = b8 ? 1 : 4;
    auto add = [&](const void* p, size_t bytes, bool out) {
      if (p != nullptr) spans.push_back({(uintptr_t)p, (uintptr_t)p + bytes, out});
    };
    add(t.p, n * 4, true);
    add(t.g, n * xsize(t.g_dtype), false);
    add(t.m, n * st, true);
    add(t.v, n * st, true);
    add(entries[i].m_scale, ns, true);
    add(entries[i].v_scale, ns, true);
    add(t.copy, n * 2, true);
  }
  // sorted by start, a span overlaps an earlier one exactly where it starts before the furthest end so far;
  // spans that are only read may share memory with each other
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.p < b.p; });
  uintptr_t end_any = 0, end_out = 0;
  for (const Span& s : spans) {
    if (s.p < (s.out ? end_any : end_out)) return WQ_EOVERLAP;
    end_any = std::max(end_any, s.end);
    if (s.out) end_out = std::max(end_out, s.end);
  }
  int rc = check_device({table});
  for (int64_t i = 0; rc == WQ_OK && i < count; ++i) {
    const wq::AdamwEntry& e = entries[i];
    if (e.n > 0) rc = check_device({e.p, e.g, e.m, e.v, e.m_scale, e.v_scale, e.copy});
  }
  for (int64_t i = 0; rc == WQ_OK && i < count; i += wq::kAdamwBatch)
    rc = launched(wq::launch_adamw_table(count, i, (int)std::min<int64_t>(wq::kAdamwBatch, count - i), chunks, state_bits,
                                         &entries[i], table, reinterpret_cast<hipStream_t>(stream)));
  return rc;
} catch (const std::bad_alloc&) {
  return WQ_EINVAL;
}

int adamw_run(int64_t count, int64_t elems, int state_bits, const void* table, const int64_t* step, const float* lr,
              double beta1, double beta2, double eps, double weight_decay, float grad_scale, uint32_t seed, void* stream) {
  if (count <= 0 || count > WQ_ADAMW_MAX_TENSORS || elems < 0 || elems > kMaxElems) return WQ_EINVAL;
  if (state_bits != 8 && state_bits != 32) return WQ_EINVAL;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return WQ_EINVAL;
  if (!(eps >= 0.0) || !std::isfinite(eps) || !(weight_decay >= 0.0) || !std::isfinite(weight_decay)) return WQ_EINVAL;
  if (any_null({table, step, lr})) return WQ_EINVAL;
  if (!all_aligned({table, step, lr})) return WQ_EALIGN;
  if (elems == 0) return WQ_OK;
  const int rc = check_device({table, step, lr});
  if (rc != WQ_OK) return rc;
  return launched(wq::launch_adamw(count, elems, state_bits, table, step, lr, beta1, beta2, eps, weight_decay, grad_scale,
                                   seed, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
