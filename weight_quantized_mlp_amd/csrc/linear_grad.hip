// Gradient of a quantised linear with respect to its input (gfx950): qlinear_backward in
// include/wqmlp_adapters.h.  One thread per element of dx, float32 sums in index order.
#include "dev_common.h"
#include "launch.h"

namespace wq {

namespace {

__global__ void linear_grad(int fmt, int M, int N, int K, const void* dy, int dyt, const uint8_t* w, const float* scale,
                            float inv, void* dx, int dxt) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)M * K) return;
  const int64_t m = i / K, k = i - m * K;
  float s = 0.f;
  for (int64_t n = 0; n < N; ++n) {
    const float g = dyt == X_F32 ? reinterpret_cast<const float*>(dy)[m * N + n]
                                 : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(dy)[m * N + n]);
    if (fmt == 0) {
      s += (g * scale[n]) * e4m3_byte_f32<0>((uint32_t)w[n * K + k]);
    } else {
      const uint8_t* rec = w + (n * (K / 64) + k / 64) * 36;
      const int kk = (int)(k & 63);
      const f32x2 v = e2m1x2_f32<0>((uint32_t)rec[4 + kk / 2]);
      s += g * ((kk & 1 ? v.y : v.x) * e4m3_byte_f32<0>((uint32_t)rec[kk / 16]) * inv);
    }
  }
  if (dxt == X_F32) reinterpret_cast<float*>(dx)[i] = s;
  else reinterpret_cast<uint16_t*>(dx)[i] = __builtin_bit_cast(uint16_t, (__bf16)s);
}

}  // namespace

size_t linear_grad_scratch_bytes(int fmt, int M, int N, int K, XType dxt) { return 0; }

hipError_t launch_linear_grad(int fmt, int M, int N, int K, const void* dy, XType dyt, const uint8_t* w, const float* scale,
                              float inv, void* ws, void* dx, XType dxt, hipStream_t st) {
  hipLaunchKernelGGL(linear_grad, dim3((unsigned)(((int64_t)M * K + 255) / 256)), dim3(256), 0, st, fmt, M, N, K, dy, dyt,
                     w, scale, inv, dx, dxt);
  return hipGetLastError();
}

}  // namespace wq
