// Shared by the kernels that multiply rows with AWQ int4 group-32 weights on the matrix cores (awq_linear.hip,
// moe_layer.hip).
//
// One MFMA (16 x 16 x 32, float16) takes 8 contraction elements from each lane: lane l holds row l % 16 of the weights and
// the octet l / 16 of the step.  Which k an octet's place stands for is free as long as both operands agree, so the weights
// stay as they are packed: a step is 4 groups of 32 k, lane quarter l / 16 holds one whole group (16 bytes of codes, one
// scale, one zero), and MFMA i of the step takes the group's dword i.
//
// Decode of a dword.  Its low nibbles, alone in their bytes, are the E4M3 codes 0 .. 15, whose values are linear: q 2^-9
// (below 8 subnormal, from 8 on of the first binade).  So two masks, a shift and four conversions of two bytes each, scaled by
// 2^9, give the 8 integers as float16, and four packed fma the weights, RN_f16(q scale + bias): 11 operations, where nibbles
// put into the mantissa of 1024 or 64 and taken out by a subtraction need 13.  Bytes hold k = 2 j (low) and 2 j + 1 (high),
// so the activations' octets are stored in the order 0 2 4 6 1 3 5 7.
#pragma once
#include "dev_common.h"
#include "launch.h"

namespace wq {

constexpr int kStepK = 128;             // contraction elements of a step: 4 groups


// 8 weights of one dword, in the order above.
__device__ __forceinline__ f16x8 awq_frag(uint32_t w, f16x2 s2, f16x2 b2) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  const f16x2 p0 = __builtin_elementwise_fma(nibbles_f16<false>(lo), s2, b2), p1 = __builtin_elementwise_fma(nibbles_f16<true>(lo), s2, b2);
  const f16x2 p2 = __builtin_elementwise_fma(nibbles_f16<false>(hi), s2, b2), p3 = __builtin_elementwise_fma(nibbles_f16<true>(hi), s2, b2);
  return f16x8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// A lane's share of one step of 16 weight rows: raw, so that every load is issued before any is used.
struct AwqStep {
  u32x4 c;
  uint32_t s, z;
};
// The scale and bias of its group, twice each; a group that is not `live` counts as zero weights.
template <int ML>
__device__ __forceinline__ void awq_meta(const AwqStep& r, bool live, f16x2& s2, f16x2& b2) {
  const _Float16 s = f16_from_bits((uint16_t)r.s);
  _Float16 b;
  if constexpr (ML == 3) b = awq_bias(r.z, s);
  else b = f16_from_bits((uint16_t)r.z);
  const _Float16 sv = live ? s : (_Float16)0.f, bv = live ? b : (_Float16)0.f;
  s2 = f16x2{sv, sv};
  b2 = f16x2{bv, bv};
}

// What float16 h left of x; nothing where h is infinite or NaN (x - h would be NaN and the infinity lose its sign).
__device__ __forceinline__ _Float16 f16_rest(float x, _Float16 h) {
  const float r = x - (float)h;
  return r == r ? (_Float16)r : (_Float16)0.f;
}

// 8 values of x -> float16 terms in octet order (0 2 4 6 1 3 5 7), scaled by 2^-e.
template <int TERMS>
__device__ __forceinline__ void octet_terms(const float* v, int e, u32x4 (&o)[TERMS]) {
  float x[8];
  _Float16 h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = ldexpf(v[j], -e);
    h[j] = (_Float16)x[j];
  }
  const u32x4 hi = {as_u32(f16x2{h[0], h[2]}), as_u32(f16x2{h[4], h[6]}), as_u32(f16x2{h[1], h[3]}), as_u32(f16x2{h[5], h[7]})};
  o[0] = hi;
  if constexpr (TERMS == 2) {
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = f16_rest(x[j], h[j]);
    const u32x4 lo = {as_u32(f16x2{h[0], h[2]}), as_u32(f16x2{h[4], h[6]}), as_u32(f16x2{h[1], h[3]}), as_u32(f16x2{h[5], h[7]})};
    o[1] = lo;
  }
}
// 8 elements of a row of x at element `at` (16-byte aligned), as loaded and as values.
template <int XT>
struct RawOctet { u32x4 v[XT == X_F32 ? 2 : 1]; };
template <int XT>
__device__ __forceinline__ RawOctet<XT> load_raw(const void* x, size_t at) {
  const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(x) + at * (XT == X_F32 ? 4 : 2));
  RawOctet<XT> r;
  r.v[0] = p[0];
  if constexpr (XT == X_F32) r.v[1] = p[1];
  return r;
}
// The same from a wave-uniform row and a 32-bit element offset in it.
template <int XT>
__device__ __forceinline__ RawOctet<XT> load_raw(const uint8_t* row, uint32_t at) {
  const u32x4* p = reinterpret_cast<const u32x4*>(row + at * (XT == X_F32 ? 4u : 2u));
  RawOctet<XT> r;
  r.v[0] = p[0];
  if constexpr (XT == X_F32) r.v[1] = p[1];
  return r;
}
template <int XT>
__device__ __forceinline__ void raw_values(const RawOctet<XT>& r, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u = r.v[0][j];
    if constexpr (XT == X_F32) {
      const uint32_t w = r.v[1][j];
      v[j] = __uint_as_float(u);
      v[4 + j] = __uint_as_float(w);
    } else if constexpr (XT == X_BF16) {
      v[2 * j] = __uint_as_float(u << 16);
      v[2 * j + 1] = __uint_as_float(u & 0xFFFF0000u);
    } else {
      const f16x2 p = as_f16x2(u);
      v[2 * j] = (float)p.x;
      v[2 * j + 1] = (float)p.y;
    }
  }
}
template <int XT>
__device__ __forceinline__ void load_octet(const void* x, size_t at, float* v) {
  raw_values<XT>(load_raw<XT>(x, at), v);
}

// 8 raw elements -> their terms scaled by 2^-e, zeros where they are not `live`.  float16 is only put in order.
template <int XT, int TERMS>
__device__ __forceinline__ void raw_terms(const RawOctet<XT>& r, int e, bool live, u32x4 (&o)[TERMS]) {
  if constexpr (XT == X_F16) {
    const uint32_t a = r.v[0][0], b = r.v[0][1], c = r.v[0][2], d = r.v[0][3];
    const u32x4 v = {__builtin_amdgcn_perm(b, a, 0x05040100), __builtin_amdgcn_perm(d, c, 0x05040100),
                     __builtin_amdgcn_perm(b, a, 0x07060302), __builtin_amdgcn_perm(d, c, 0x07060302)};
    const u32x4 zero = {0, 0, 0, 0};
    o[0] = live ? v : zero;
  } else {
    float v[8];
    raw_values<XT>(r, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = live ? v[j] : 0.f;
    octet_terms<TERMS>(v, e, o);
  }
}
template <int XT>
__device__ __forceinline__ float octet_max(const RawOctet<XT>& r) {
  float v[8], m = 0.f;
  raw_values<XT>(r, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(v[j]));
  return m;
}
// A wave's 64 octets -> terms, scaled by the power of two that is returned.
template <int XT, int TERMS>
__device__ __forceinline__ float wave_terms(const RawOctet<XT>& r, bool live, u32x4 (&o)[TERMS]) {
  const int e = XT == X_F16 ? 0 : f16_row_exp(wave64_max(live ? octet_max<XT>(r) : 0.f));
  raw_terms<XT, TERMS>(r, e, live, o);
  return ldexpf(1.f, e);
}

// float32 rows take two float16 terms (their products' sum is off by 2^-22 of an element or 2^-39 of its row's largest), bfloat16
// ones fit into one after the scaling (down to 2^-39 of the row's largest), float16 ones are taken as they are.
inline int awq_terms(XType xt) { return xt == X_F32 ? 2 : 1; }

}  // namespace wq
