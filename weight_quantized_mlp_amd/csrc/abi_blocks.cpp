// C ABI of the block calls (declarations and contracts: include/wqmlp_blocks.h).
// The checks come in the two phases of abi.cpp: arithmetic on the arguments, then the device.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/wqmlp_blocks.h"
#include "abi_common.h"
#include "launch.h"

namespace {

using namespace wq::abi;

bool is_float(int dt) { return dt == WQ_F32 || dt == WQ_BF16 || dt == WQ_F16; }
wq::XType xtype(int dt) { return dt == WQ_F32 ? wq::X_F32 : (dt == WQ_BF16 ? wq::X_BF16 : wq::X_F16); }

bool is_grad(int dt) { return dt == WQ_F32 || dt == WQ_BF16; }

bool awq_shape_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && M <= kMaxDim && N > 0 && N <= kMaxDim && K > 0 && K <= kMaxDim && K % 32 == 0 &&
         M * (N > K ? N : K) <= kMaxElems;
}

bool moe_shape_ok(int64_t M, int64_t E, int64_t topk, int64_t H, int64_t I) {
  return M >= 0 && M <= WQ_MOE_MAX_TOKENS && E > 0 && E <= kMaxDim && topk > 0 && topk <= WQ_MOE_MAX_TOPK && H > 0 &&
         H <= WQ_MOE_MAX_WIDTH && H % 32 == 0 && I > 0 && I <= WQ_MOE_MAX_WIDTH && I % 32 == 0 && E <= kMaxElems / H &&
         E <= kMaxElems / (2 * I);
}

// A gate of its own for every row of none has no rows.
bool norm_shape_ok(int64_t M, int64_t H, int64_t G) {
  return M >= 0 && M <= kMaxDim && H > 0 && H <= kMaxDim && H % 8 == 0 && G >= 0 && G <= kMaxDim && (G == 0 ? M == 0 : M % G == 0) &&
         M * H <= kMaxElems && G * H <= kMaxElems;
}

// Types of the tensors that are there, and the constants.
bool norm_args_ok(const void* y, int yt, int ht, const void* post, const void* pre, int wt, int xt, const void* gate,
                  int64_t G, int gt, float alpha, float offset, float eps) {
  if (!is_float(ht) || (y != nullptr && !is_float(yt))) return false;
  if ((post != nullptr || pre != nullptr) && !is_float(wt)) return false;
  if (pre != nullptr && !is_float(xt)) return false;
  if (gate == nullptr ? G != 1 : !is_float(gt)) return false;
  if (y == nullptr && (post != nullptr || gate != nullptr)) return false;
  if (y == nullptr && pre == nullptr) return false;
  return std::isfinite(alpha) && std::isfinite(offset) && eps >= 0.f && std::isfinite(eps);
}

wq::BlockNorm norm_of(const void* h, int ht, const void* y, int yt, const void* post, const void* pre, int wt, const void* gate,
                      int64_t G, int gt, float alpha, float offset, float eps) {
  return {h, y, post, pre, gate, xtype(ht), xtype(yt), xtype(wt), xtype(gt), (int)G, alpha, offset, eps};
}

size_t bytes_of(const void* p, int64_t n, int dt) { return p == nullptr ? 0 : (size_t)n * xsize(dt); }

}  // namespace

extern "C" {

size_t awq_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_dtype) {
  if (!awq_shape_ok(M, N, K) || !is_float(x_dtype)) return 0;
  return wq::awq_linear_scratch_bytes((int)M, (int)N, (int)K, xtype(x_dtype));
}

int awq_linear_run(int64_t M, int64_t N, int64_t K, const void* x, int x_dtype, const void* bank, int meta_layout,
                   void* workspace, size_t workspace_bytes, float* y, void* stream) {
  if (!awq_shape_ok(M, N, K) || !is_float(x_dtype) || (meta_layout != 3 && meta_layout != 4)) return WQ_EINVAL;
  if (bank == nullptr) return WQ_EINVAL;
  if (M == 0) return WQ_OK;
  if (any_null({x, y})) return WQ_EINVAL;
  if (!all_aligned({x, bank, workspace, y})) return WQ_EALIGN;
  const size_t need = awq_linear_workspace_bytes(M, N, K, x_dtype);
  if (need && (workspace == nullptr || workspace_bytes < need)) return WQ_EWORKSPACE;
  if (any_overlap({{y, (size_t)M * N * 4}, {workspace, need}},
                  {{x, (size_t)M * K * xsize(x_dtype)}, {bank, awq_bank_bytes(1, N, K, meta_layout)}}))
    return WQ_EOVERLAP;
  const int rc = check_device({x, bank, need ? workspace : nullptr, y});
  if (rc != WQ_OK) return rc;
  return launched(wq::launch_awq_linear((int)M, (int)N, (int)K, x, xtype(x_dtype), static_cast<const uint8_t*>(bank), meta_layout,
                                        workspace, y, reinterpret_cast<hipStream_t>(stream)));
}

size_t awq_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int dy_dtype, int dx_dtype) {
  if (!awq_shape_ok(M, N, K) || !is_grad(dy_dtype) || !is_grad(dx_dtype)) return 0;
  return wq::awq_linear_grad_scratch_bytes((int)M, (int)N, (int)K, xtype(dy_dtype), xtype(dx_dtype));
}

int awq_linear_backward(int64_t M, int64_t N, int64_t K, const void* dy, int dy_dtype, const void* bank, int meta_layout,
                        void* workspace, size_t workspace_bytes, void* dx, int dx_dtype, void* stream) {
  if (!awq_shape_ok(M, N, K) || !is_grad(dy_dtype) || !is_grad(dx_dtype) || (meta_layout != 3 && meta_layout != 4)) return WQ_EINVAL;
  if (bank == nullptr) return WQ_EINVAL;
  if (M == 0) return WQ_OK;
  if (any_null({dy, dx})) return WQ_EINVAL;
  if (!all_aligned({dy, bank, workspace, dx})) return WQ_EALIGN;
  const size_t need = awq_linear_backward_workspace_bytes(M, N, K, dy_dtype, dx_dtype);
  if (need && (workspace == nullptr || workspace_bytes < need)) return WQ_EWORKSPACE;
  if (any_overlap({{dx, (size_t)M * K * xsize(dx_dtype)}, {workspace, need}},
                  {{dy, (size_t)M * N * xsize(dy_dtype)}, {bank, awq_bank_bytes(1, N, K, meta_layout)}}))
    return WQ_EOVERLAP;
  const int rc = check_device({dy, bank, need ? workspace : nullptr, dx});
  if (rc != WQ_OK) return rc;
  return launched(wq::launch_awq_linear_grad((int)M, (int)N, (int)K, dy, xtype(dy_dtype), static_cast<const uint8_t*>(bank),
                                             meta_layout, workspace, dx, xtype(dx_dtype), reinterpret_cast<hipStream_t>(stream)));
}

size_t moe_awq_workspace_bytes(int64_t M, int64_t E, int64_t topk, int64_t H, int64_t I) {
  if (!moe_shape_ok(M, E, topk, H, I)) return 0;
  return wq::moe_awq_scratch_bytes((int)M, (int)E, (int)topk, (int)H, (int)I);
}

int moe_awq_run(int64_t M, int64_t E, int64_t topk, int64_t H, int64_t I, const void* x, int x_dtype, const void* router,
                int router_dtype, int32_t* ids, float* weights, const void* w13_bank, const void* w2_bank, int meta_layout,
                void* workspace, size_t workspace_bytes, void* out, int out_dtype, int flags, void* stream) {
  if (!moe_shape_ok(M, E, topk, H, I) || !is_float(x_dtype) || !is_float(out_dtype)) return WQ_EINVAL;
  if (meta_layout != 3 && meta_layout != 4) return WQ_EINVAL;
  if (router == nullptr ? flags != 0 : (!is_float(router_dtype) || topk > E || (flags & ~WQ_MOE_RENORM) != 0)) return WQ_EINVAL;
  if (any_null({w13_bank, w2_bank})) return WQ_EINVAL;
  if (M == 0) return WQ_OK;
  if (any_null({x, ids, weights, out})) return WQ_EINVAL;
  if (!all_aligned({x, router, ids, weights, w13_bank, w2_bank, workspace, out})) return WQ_EALIGN;
  const size_t need = moe_awq_workspace_bytes(M, E, topk, H, I);
  if (need && (workspace == nullptr || workspace_bytes < need)) return WQ_EWORKSPACE;
  const Rng rx{x, (size_t)M * H * xsize(x_dtype)}, ri{ids, (size_t)M * topk * 4}, rw{weights, (size_t)M * topk * 4};
  const Rng rr{router, router ? (size_t)E * H * xsize(router_dtype) : 0};
  const Rng r13{w13_bank, awq_bank_bytes(E, 2 * I, H, meta_layout)}, r2{w2_bank, awq_bank_bytes(E, H, I, meta_layout)};
  const Rng ro{out, (size_t)M * H * xsize(out_dtype)}, rs{workspace, need};
  if (router != nullptr ? any_overlap({ro, rs, ri, rw}, {rx, rr, r13, r2}) : any_overlap({ro, rs}, {rx, ri, rw, r13, r2}))
    return WQ_EOVERLAP;
  const int rc = check_device({x, router, ids, weights, w13_bank, w2_bank, need ? workspace : nullptr, out});
  if (rc != WQ_OK) return rc;
  return launched(wq::launch_moe_awq((int)M, (int)E, (int)topk, (int)H, (int)I, x, xtype(x_dtype), router, xtype(router_dtype),
                                     (flags & WQ_MOE_RENORM) != 0, ids, weights, static_cast<const uint8_t*>(w13_bank),
                                     static_cast<const uint8_t*>(w2_bank), meta_layout, workspace, out, xtype(out_dtype),
                                     reinterpret_cast<hipStream_t>(stream)));
}

int block_norm_run(int64_t M, int64_t H, const void* h, int h_dtype, const void* y, int y_dtype, const void* post,
                   const void* pre, int w_dtype, const void* gate, int64_t G, int g_dtype, float alpha, float offset,
                   float eps, void* h_out, void* x, int x_dtype, void* stream) {
  if (!norm_shape_ok(M, H, G)) return WQ_EINVAL;
  if (M == 0) {   // an empty tensor's address is NULL: which tensors there are cannot be told
    return is_float(h_dtype) ? WQ_OK : WQ_EINVAL;
  }
  if (!norm_args_ok(y, y_dtype, h_dtype, post, pre, w_dtype, x_dtype, gate, G, g_dtype, alpha, offset, eps)) return WQ_EINVAL;
  if (h == nullptr || (y != nullptr) != (h_out != nullptr) || (pre != nullptr) != (x != nullptr)) return WQ_EINVAL;
  if (!all_aligned({h, y, post, pre, gate, h_out, x})) return WQ_EALIGN;
  const size_t nh = (size_t)M * H * xsize(h_dtype);
  if (any_overlap({{h_out, h_out ? nh : 0}, {x, bytes_of(x, M * H, x_dtype)}},
                  {{h, h == h_out ? 0 : nh}, {y, bytes_of(y, M * H, y_dtype)}, {post, bytes_of(post, H, w_dtype)},
                   {pre, bytes_of(pre, H, w_dtype)}, {gate, bytes_of(gate, G * H, g_dtype)}}))
    return WQ_EOVERLAP;
  const int rc = check_device({h, y, post, pre, gate, h_out, x});
  if (rc != WQ_OK) return rc;
  return launched(wq::launch_block_norm((int)M, (int)H,
                                        norm_of(h, h_dtype, y, y_dtype, post, pre, w_dtype, gate, G, g_dtype, alpha, offset, eps),
                                        h_out, x, xtype(x_dtype), reinterpret_cast<hipStream_t>(stream)));
}

size_t block_norm_backward_workspace_bytes(int64_t M, int64_t H, int64_t G) {
  if (!norm_shape_ok(M, H, G)) return 0;
  return wq::block_norm_grad_scratch_bytes((int)M, (int)H, (int)G);
}

int block_norm_backward(int64_t M, int64_t H, const void* h, int h_dtype, const void* y, int y_dtype, const void* dh,
                        const void* dx, int x_dtype, const void* post, const void* pre, int w_dtype, const void* gate,
                        int64_t G, int g_dtype, float alpha, float offset, float eps, void* workspace,
                        size_t workspace_bytes, void* dh_in, void* dy, float* dpost, float* dgate, float* dpre,
                        void* stream) {
  if (!norm_shape_ok(M, H, G)) return WQ_EINVAL;
  if (M == 0) {   // the weights' gradients are zero; the rows' tensors are empty
    if (!is_float(h_dtype)) return WQ_EINVAL;
    h = y = dh = dx = nullptr;
    dh_in = dy = nullptr;
    if (dpost == nullptr && dgate == nullptr && dpre == nullptr) return WQ_OK;
  } else {
    if (!norm_args_ok(y, y_dtype, h_dtype, post, pre, w_dtype, x_dtype, gate, G, g_dtype, alpha, offset, eps)) return WQ_EINVAL;
    if (h == nullptr || (pre != nullptr) != (dx != nullptr)) return WQ_EINVAL;
    if (dh_in == nullptr && dy == nullptr && dpost == nullptr && dgate == nullptr && dpre == nullptr) return WQ_EINVAL;
    if (y == nullptr && (dy != nullptr || dpost != nullptr || dgate != nullptr)) return WQ_EINVAL;
  }
  if ((dpost != nullptr && post == nullptr) || (dgate != nullptr && gate == nullptr) || (dpre != nullptr && pre == nullptr))
    return WQ_EINVAL;
  if (!all_aligned({h, y, dh, dx, post, pre, gate, workspace, dh_in, dy, dpost, dgate, dpre})) return WQ_EALIGN;
  const size_t need = block_norm_backward_workspace_bytes(M, H, G);
  if (need && (workspace == nullptr || workspace_bytes < need)) return WQ_EWORKSPACE;
  const size_t nh = (size_t)M * H * xsize(h_dtype);
  if (any_overlap({{dh_in, dh_in ? nh : 0}, {dy, bytes_of(dy, M * H, y_dtype)}, {dpost, dpost ? (size_t)H * 4 : 0},
                   {dgate, dgate ? (size_t)G * H * 4 : 0}, {dpre, dpre ? (size_t)H * 4 : 0}, {workspace, need}},
                  {{h, h ? nh : 0}, {y, bytes_of(y, M * H, y_dtype)}, {dh, dh == nullptr || dh == dh_in ? 0 : nh},
                   {dx, bytes_of(dx, M * H, x_dtype)}, {post, bytes_of(post, H, w_dtype)}, {pre, bytes_of(pre, H, w_dtype)},
                   {gate, bytes_of(gate, G * H, g_dtype)}}))
    return WQ_EOVERLAP;
  const int rc = check_device({h, y, dh, dx, post, pre, gate, need ? workspace : nullptr, dh_in, dy, dpost, dgate, dpre});
  if (rc != WQ_OK) return rc;
  return launched(wq::launch_block_norm_grad(
      (int)M, (int)H, norm_of(h, h_dtype, y, y_dtype, post, pre, w_dtype, gate, G, g_dtype, alpha, offset, eps), dh, dx,
      xtype(x_dtype), workspace, dh_in, dy, dpost, dgate, dpre, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
