// AdamW over many tensors in one launch (gfx950).
//
// Mathematics and state forms: adamw_run in include/wqmlp_adapters.h.  The step is a stream: 28 bytes per
// element with float32 states and gradients (p, m, v read and written, g read), 16 with 8-bit states, plus
// 2 for a 16-bit copy, against some 30 (8-bit states: 80) ALU operations, so HBM bounds it and one pass
// over every array is the whole plan.  The tensors are cut into chunks of kChunk elements, numbered through
// all tensors; a workgroup takes a chunk (in huge tables a run of them), finds its tensor with a 256-way
// search of the table's chunk starts and walks on from there, so one launch serves any number of tensors
// of any sizes (chosen against 2048 workgroups with a run of chunks each at 800 us to 837 for 178M
// elements with float32 states, 264 to 285 for 83M with 8-bit states; over several cards 800-863, 5.4-5.8
// TB/s, and 263-282).  A wave takes 256
// consecutive elements at a time, 4 per lane: 16-byte accesses to the float32 arrays, 4-byte accesses to
// the codes, and a block's scale is one wave maximum.
#include <algorithm>

#include "dev_common.h"
#include "launch.h"

namespace wq {

namespace {

constexpr int kChunk = 4096;

struct AdamwBatch {
  AdamwEntry e[kAdamwBatch];
};

__global__ void adamw_table_kernel(uint8_t* table, int64_t count, int64_t first, int n, int64_t total, int bits,
                                   AdamwBatch b) {
  const int i = threadIdx.x;
  int64_t* head = reinterpret_cast<int64_t*>(table);
  if (first == 0 && i == 0) {
    head[0] = count;
    head[1] = total;
    head[2] = bits;
    head[kAdamwHead + count] = total;
  }
  if (i < n) {
    head[kAdamwHead + first + i] = b.e[i].chunk0;
    reinterpret_cast<AdamwEntry*>(table + adamw_entries_offset(count))[first + i] = b.e[i];
  }
}

// 32-bit integer mix (two rounds of multiply and xor-shift; the constants are those that C. Wellons found by search and
// published in "Prospecting for Hash Functions", 2018).
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x7FEB352Du;
  h ^= h >> 15;
  h *= 0x846CA68Bu;
  return h ^ (h >> 16);
}

// beta^t by repeated squaring in double.  Every squaring doubles the relative error, which ends near t 2^-53; that of
// 1 - beta^t is then at most 2^-53 / (1 - beta), since t beta^t / (1 - beta^t) < 1 / (1 - beta): 2^-40 for 0.9999.
__device__ __forceinline__ double pow_int(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

// Square root within one unit.  The instruction takes subnormal operands as zero, whose roots are ordinary numbers: small
// operands go through it scaled.
__device__ __forceinline__ float root(float x) {
  const bool small = x < 0x1p-96f;
  return __builtin_amdgcn_sqrtf(small ? x * 0x1p64f : x) * (small ? 0x1p-32f : 1.0f);
}

__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  v = fmaxf(v, dpp_f32<0x140>(v));
  const int b = __builtin_bit_cast(int, v);
  const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return fmaxf(fmaxf(r0, r1), fmaxf(r2, r3));
}

// Smallest e in [-100, 100] with amax <= 0.875 * 2^half * 2^e; 0 for a zero amax.
__device__ __forceinline__ int block_exp(float amax, int half) {
  if (!(amax > 0.f)) return 0;
  int p;
  const float f = frexpf(amax, &p);
  const int e = p - half + (f > 0.875f ? 1 : 0);
  return e < -100 ? -100 : (e > 100 ? 100 : e);
}

// |x| already divided by the block scale -> stochastically rounded magnitude on the code's grid (MANT mantissa
// bits, smallest normal 2^EMIN, from `least` to MAXV), NaN if x is not finite.  r: 16 random bits.
template <int MANT, int EMIN>
__device__ __forceinline__ float round_code(float x, uint32_t r, float least, float maxv) {
  constexpr int DROP = 23 - MANT;
  const float mag = fabsf(x);
  const uint32_t up = ((__float_as_uint(mag) + (r << (DROP - 16))) >> DROP) << DROP;
  constexpr float kMin = EMIN == -6 ? 0x1p-6f : 0x1p-14f, kStep = EMIN == -6 ? 0x1p-9f : 0x1p-16f;
  static_assert((EMIN == -6 && MANT == 3) || (EMIN == -14 && MANT == 2), "E4M3 or E5M2");
  const uint32_t fixed = (uint32_t)(fminf(mag, kMin) * (65536.0f / kStep));   // below 2^20: exact multiples of 2^-16 steps
  const float sub = (float)((fixed + r) >> 16) * kStep;
  float q = mag < kMin ? sub : __uint_as_float(up);
  q = fminf(fmaxf(q, least), maxv);
  q = mag <= 3.4028235e38f ? q : __uint_as_float(0x7FC00000u);
  return copysignf(q, x);
}

__device__ __forceinline__ uint32_t round_bf16(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ uint32_t round_f16(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v);
}

struct AdamwHyper {
  float beta1, omb1, beta2, omb2, eps, grad_scale;   // omb = 1 - beta
  double b1, b2;
  float decay;
  uint32_t seed;
};

// One vector load or store, NT: with the non-temporal hint.
template <bool NT, typename T>
__device__ __forceinline__ T vload(const T* p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool NT, typename T>
__device__ __forceinline__ void vstore(T v, T* p) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}
// Four consecutive elements at index i (i a multiple of 4); elements at n and beyond read as 0 / not written.
template <bool NT>
__device__ __forceinline__ void load4(const float* a, int64_t i, int64_t n, float* v) {
  if (i + 4 <= n) {
    const f32x4 t = vload<NT>(reinterpret_cast<const f32x4*>(a + i));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = t[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < n ? a[i + j] : 0.f;
  }
}
template <bool NT>
__device__ __forceinline__ void load4(const uint16_t* a, int64_t i, int64_t n, float* v) {   // bfloat16
  if (i + 4 <= n) {
    const u32x2 t = vload<NT>(reinterpret_cast<const u32x2*>(a + i));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      v[2 * j] = __uint_as_float(t[j] << 16);
      v[2 * j + 1] = __uint_as_float(t[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < n ? bf16_bits_to_f32(a[i + j]) : 0.f;
  }
}
template <bool NT>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* a, int64_t i, int64_t n) {
  if (i + 4 <= n) return vload<NT>(reinterpret_cast<const uint32_t*>(a + i));
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) w |= (uint32_t)a[i + j] << (8 * j);
  return w;
}
template <bool NT>
__device__ __forceinline__ void store4(float* a, int64_t i, int64_t n, const float* v) {
  if (i + 4 <= n) {
    vstore<NT>(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(a + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) a[i + j] = v[j];
  }
}
template <bool NT>
__device__ __forceinline__ void store_codes(uint8_t* a, int64_t i, int64_t n, uint32_t w) {
  if (i + 4 <= n) {
    vstore<NT>(w, reinterpret_cast<uint32_t*>(a + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) a[i + j] = (uint8_t)(w >> (8 * j));
  }
}

template <int BITS, bool NT>
__global__ void __launch_bounds__(256) adamw_kernel(const uint8_t* __restrict__ table, const int64_t* __restrict__ step_p,
                                                    const float* __restrict__ lr_p, AdamwHyper h) {
  const int64_t* head = reinterpret_cast<const int64_t*>(table);
  const int64_t count = head[0], total = head[1];
  if ((head[2] & 255) != BITS) return;   // a table of the other state form: nothing is touched
  const float least_v = (head[2] & kAdamwKeepV) != 0 ? 0x1p-16f : 0.f;   // v's smallest code, where a positive v keeps one
  const int64_t* chunk0 = head + kAdamwHead;
  const AdamwEntry* entries = reinterpret_cast<const AdamwEntry*>(table + adamw_entries_offset(count));
  const int64_t per = total <= gridDim.x ? 1 : (total + gridDim.x - 1) / gridDim.x;   // a 64-bit division is 140 instructions
  int64_t c = (int64_t)blockIdx.x * per;
  const int64_t c1 = c + per < total ? c + per : total;
  if (c >= c1) return;
  // tensor of chunk c: the last with chunk0 <= c (empty tensors share a start with their successor), by 256-way steps: one for
  // up to 256 tensors, three for the most a table holds
  int64_t t = 0;
  for (int64_t span = count;;) {
    const int64_t stride = (span + 255) / 256, i = threadIdx.x * stride;
    const int64_t below = __syncthreads_count(i < span && chunk0[t + i] <= c) - 1;   // the first always is
    t += below * stride;
    if (stride == 1) break;
    span = min(stride, span - below * stride);
  }
  const int64_t step = *step_p;
  const float lr = *lr_p;
  const float ibc1 = (float)(1.0 / (1.0 - pow_int(h.b1, step))), ibc2 = (float)(1.0 / (1.0 - pow_int(h.b2, step)));
  const float keep = 1.0f - lr * h.decay;
  const uint32_t key0 = mix32(h.seed + 0x9E3779B9u * (uint32_t)step);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  for (; c < c1; ++c) {
    while (c >= chunk0[t + 1]) ++t;
    const AdamwEntry e = entries[t];
    const int64_t n = e.n;
    const int64_t base = (c - e.chunk0) * kChunk;
    const uint32_t key = mix32(key0 + (uint32_t)t);
#pragma unroll
    for (int q = 0; q < kChunk / 1024; ++q) {
      const int64_t b0 = base + 1024 * q + 256 * wave;   // this wave's block
      if (b0 >= n) break;
      const int64_t i = b0 + 4 * lane;
      float p[4], g[4], m[4], v[4];
      load4<NT>(e.p, i, n, p);
      if (e.g_dtype == 0) load4<NT>(reinterpret_cast<const float*>(e.g), i, n, g);
      else load4<NT>(reinterpret_cast<const uint16_t*>(e.g), i, n, g);
      if constexpr (BITS == 32) {
        load4<NT>(reinterpret_cast<const float*>(e.m), i, n, m);
        load4<NT>(reinterpret_cast<const float*>(e.v), i, n, v);
      } else {
        const uint32_t mc = load_codes<NT>(reinterpret_cast<const uint8_t*>(e.m), i, n);
        const uint32_t vc = load_codes<NT>(reinterpret_cast<const uint8_t*>(e.v), i, n);
        const float ms = e.m_scale[b0 >> 8], vs = e.v_scale[b0 >> 8];
        const f32x2 m0 = e4m3x2_f32<false>(mc), m1 = e4m3x2_f32<true>(mc);
        const f32x2 v0 = __builtin_amdgcn_cvt_pk_f32_bf8(vc, false), v1 = __builtin_amdgcn_cvt_pk_f32_bf8(vc, true);
        m[0] = m0.x * ms; m[1] = m0.y * ms; m[2] = m1.x * ms; m[3] = m1.y * ms;
        v[0] = v0.x * vs; v[1] = v0.y * vs; v[2] = v1.x * vs; v[3] = v1.y * vs;
      }
      {
        // every product and sum of the state update is rounded by itself, so that the codes do not depend
        // on which of them a compiler fuses
#pragma clang fp contract(off)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float gj = g[j] * h.grad_scale;
          const float mj = m[j] * h.beta1, dj = gj * h.omb1;
          m[j] = mj + dj;
          const float g2 = gj * gj;
          const float vj = v[j] * h.beta2, wj = g2 * h.omb2;
          v[j] = vj + wj;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float d = root(v[j] * ibc2) + h.eps;
        p[j] = p[j] * keep - lr * ((m[j] * ibc1) * __builtin_amdgcn_rcpf(d));
      }
      store4<NT>(e.p, i, n, p);
      if (e.copy != nullptr) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = e.copy_dtype == 1 ? round_bf16(p[j]) : round_f16(p[j]);
        uint16_t* o = reinterpret_cast<uint16_t*>(e.copy);
        if (i + 4 <= n) {
          vstore<NT>(u32x2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)}, reinterpret_cast<u32x2*>(o + i));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i + j < n) o[i + j] = (uint16_t)w[j];
        }
      }
      if constexpr (BITS == 32) {
        store4<NT>(reinterpret_cast<float*>(e.m), i, n, m);
        store4<NT>(reinterpret_cast<float*>(e.v), i, n, v);
      } else {
        // a state that is not finite has no say in its block's scale
        const float am = fmaxf(fmaxf(finite_abs(m[0]), finite_abs(m[1])), fmaxf(finite_abs(m[2]), finite_abs(m[3])));
        const float av = fmaxf(fmaxf(finite_abs(v[0]), finite_abs(v[1])), fmaxf(finite_abs(v[2]), finite_abs(v[3])));
        const int em = block_exp(wave_max(am), 9), ev = block_exp(wave_max(av), 16);
        const float im = ldexpf(1.0f, -em), iv = ldexpf(1.0f, -ev);
        if (lane == 0) {
          e.m_scale[b0 >> 8] = ldexpf(1.0f, em);
          e.v_scale[b0 >> 8] = ldexpf(1.0f, ev);
        }
        float qm[4], qv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t r = mix32(key + 0x9E3779B9u * (uint32_t)(i + j));
          qm[j] = round_code<3, -6>(m[j] * im, r & 0xFFFFu, 0.f, 448.f);
          qv[j] = round_code<2, -14>(v[j] * iv, r >> 16, v[j] > 0.f ? least_v : 0.f, 57344.f);
        }
        int cm = __builtin_amdgcn_cvt_pk_fp8_f32(qm[0], qm[1], 0, false);
        cm = __builtin_amdgcn_cvt_pk_fp8_f32(qm[2], qm[3], cm, true);
        int cv = __builtin_amdgcn_cvt_pk_bf8_f32(qv[0], qv[1], 0, false);
        cv = __builtin_amdgcn_cvt_pk_bf8_f32(qv[2], qv[3], cv, true);
        store_codes<NT>(reinterpret_cast<uint8_t*>(e.m), i, n, (uint32_t)cm);
        store_codes<NT>(reinterpret_cast<uint8_t*>(e.v), i, n, (uint32_t)cv);
      }
    }
  }
}

}  // namespace

int64_t adamw_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

hipError_t launch_adamw_table(int64_t count, int64_t first, int n, int64_t total, int bits, const AdamwEntry* e,
                              void* table, hipStream_t st) {
  AdamwBatch b{};
  for (int i = 0; i < n; ++i) b.e[i] = e[i];
  hipLaunchKernelGGL(adamw_table_kernel, dim3(1), dim3(64), 0, st, reinterpret_cast<uint8_t*>(table), count, first, n,
                     total, bits, b);
  return hipGetLastError();
}

hipError_t launch_adamw(int64_t count, int64_t elems, int bits, const void* table, const int64_t* step, const float* lr,
                        double beta1, double beta2, double eps, double weight_decay, float grad_scale, uint32_t seed,
                        hipStream_t st) {
  // The root of any v is 0 or above 2^-75, so a positive eps below 2^-126 matters only where v is 0: there it keeps
  // 0 / eps at 0, which a subnormal would not (the reciprocal instruction takes one as zero).
  const float eps32 = eps > 0.0 ? std::max((float)eps, 0x1p-126f) : 0.f;
  const AdamwHyper h{(float)beta1, (float)(1.0 - beta1), (float)beta2, (float)(1.0 - beta2), eps32, grad_scale,
                     beta1, beta2, (float)weight_decay, seed};
  const int64_t chunks = adamw_chunks(elems) + count;   // at least the table's number
  const unsigned grid = (unsigned)(chunks < (1 << 22) ? chunks : (1 << 22));
  // Tables beyond the last-level cache stream with the non-temporal hint, smaller ones find last step's
  // states there.  us with and without it, a bfloat16 gradient written just before: float32 states 16M
  // elements 92 and 77, 24M 134 and 143, 64M 332 and 370; 8-bit 53 and 46, 78 and 81, 193 and 221.
  const bool nt = elems >= ((int64_t)20 << 20);
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, st, reinterpret_cast<const uint8_t*>(table), step, lr, h);
  };
  if (bits == 8) nt ? launch(adamw_kernel<8, true>) : launch(adamw_kernel<8, false>);
  else nt ? launch(adamw_kernel<32, true>) : launch(adamw_kernel<32, false>);
  return hipGetLastError();
}

}  // namespace wq
