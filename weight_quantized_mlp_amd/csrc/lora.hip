// Low-rank adapters beside a shared projection, forward and backward (gfx950): lora_run and lora_backward
// in include/wqmlp_adapters.h.  One thread per output element, float32 sums in index order.
#include "dev_common.h"
#include "launch.h"

namespace wq {

namespace {

// Element i of an array of type xt (X_F32, X_BF16, X_F16) as float32.
__device__ __forceinline__ float elem(const void* p, int xt, int64_t i) {
  if (xt == X_F32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
  return xt == X_BF16 ? bf16_bits_to_f32(b) : (float)f16_from_bits(b);
}

// t[m,r] = f sum_k x[m,k] w[e][r sr + k sk], e = ids[m], f = scale[e] or 1 (scale null).
__global__ void lora_shrink(int M, int K, int E, int R, const void* x, int xt, const void* w, int wt, int64_t sr,
                            int64_t sk, const float* scale, const int32_t* ids, float* t) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)M * R) return;
  const int64_t m = i / R, r = i - m * R;
  const int e = ids[m];
  float s = 0.f;
  if (e >= 0 && e < E) {
    for (int k = 0; k < K; ++k) s += elem(x, xt, m * K + k) * elem(w, wt, (int64_t)e * R * K + r * sr + k * sk);
    if (scale) s *= scale[e];
  }
  t[i] = s;
}

// out[m,n] = base[m,n] + f sum_r t[m,r] w[e][n sn + r sr].
__global__ void lora_expand(int M, int N, int E, int R, const float* t, const void* w, int wt, int64_t sn, int64_t sr,
                            const float* scale, const int32_t* ids, const void* base, void* out, int ot) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)M * N) return;
  const int64_t m = i / N, n = i - m * N;
  const int e = ids[m];
  float v = base ? elem(base, ot, i) : 0.f;
  if (e >= 0 && e < E) {
    float s = 0.f;
    for (int r = 0; r < R; ++r) s += t[m * R + r] * elem(w, wt, (int64_t)e * R * N + n * sn + r * sr);
    v += scale ? s * scale[e] : s;
  }
  if (ot == X_F32) reinterpret_cast<float*>(out)[i] = v;
  else if (ot == X_BF16) reinterpret_cast<uint16_t*>(out)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
  else reinterpret_cast<uint16_t*>(out)[i] = __builtin_bit_cast(uint16_t, (_Float16)v);
}

// g[e][r sr + d sd] = f sum_{m: ids[m] = e} u[m,r] v[m,d].
__global__ void lora_outer(int M, int D, int E, int R, const float* u, const void* v, int vt, const float* scale,
                           const int32_t* ids, float* g, int64_t sr, int64_t sd) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)E * R * D) return;
  const int64_t e = i / ((int64_t)R * D), j = i - e * R * D, r = j / D, d = j - r * D;
  float s = 0.f;
  for (int64_t m = 0; m < M; ++m)
    if (ids[m] == e) s += (scale ? u[m * R + r] * scale[e] : u[m * R + r]) * elem(v, vt, m * D + d);
  g[e * R * D + r * sr + d * sd] = s;
}

inline dim3 grid_for(int64_t n) { return dim3((unsigned)((n + 255) / 256)); }

}  // namespace

size_t lora_scratch_bytes(int M, int K, int N, int E, int R, bool backward) {
  return (size_t)M * R * 4 * (backward ? 2 : 1);
}

hipError_t launch_lora(int M, int K, int N, int E, int R, const void* x, XType xt, const void* a, const void* b, XType wt,
                       const float* scale, const int32_t* ids, const float* y, void* ws, float* out, hipStream_t st) {
  float* t = reinterpret_cast<float*>(ws);
  hipLaunchKernelGGL(lora_shrink, grid_for((int64_t)M * R), dim3(256), 0, st, M, K, E, R, x, xt, a, wt, (int64_t)K, 1,
                     nullptr, ids, t);
  hipLaunchKernelGGL(lora_expand, grid_for((int64_t)M * N), dim3(256), 0, st, M, N, E, R, t, b, wt, (int64_t)R, 1, scale,
                     ids, y, out, X_F32);
  return hipGetLastError();
}

hipError_t launch_lora_backward(int M, int K, int N, int E, int R, const void* dy, XType dyt, const void* x, XType xt,
                                const void* a, const void* b, XType wt, const float* scale, const int32_t* ids,
                                const void* dx0, XType dxt, void* ws, void* dx, float* da, float* db, hipStream_t st) {
  float* t = reinterpret_cast<float*>(ws);
  float* dt = t + (size_t)M * R;
  if (M > 0) {
    hipLaunchKernelGGL(lora_shrink, grid_for((int64_t)M * R), dim3(256), 0, st, M, K, E, R, x, xt, a, wt, (int64_t)K, 1,
                       nullptr, ids, t);
    hipLaunchKernelGGL(lora_shrink, grid_for((int64_t)M * R), dim3(256), 0, st, M, N, E, R, dy, dyt, b, wt, 1, (int64_t)R,
                       scale, ids, dt);
  }
  if (db)
    hipLaunchKernelGGL(lora_outer, grid_for((int64_t)E * R * N), dim3(256), 0, st, M, N, E, R, t, dy, dyt, scale, ids, db,
                       1, (int64_t)R);
  if (da)
    hipLaunchKernelGGL(lora_outer, grid_for((int64_t)E * R * K), dim3(256), 0, st, M, K, E, R, dt, x, xt, nullptr, ids, da,
                       (int64_t)K, 1);
  if (dx && M > 0)
    hipLaunchKernelGGL(lora_expand, grid_for((int64_t)M * K), dim3(256), 0, st, M, K, E, R, dt, a, wt, 1, (int64_t)K,
                       nullptr, ids, dx0, dx, dxt);
  return hipGetLastError();
}

}  // namespace wq
