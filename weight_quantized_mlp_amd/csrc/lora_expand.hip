// Low-rank adapters, the product back from the rank (gfx950): out[m,n] = base[m,n] + scale[e] sum_r t[m,r] w[e][n,r],
// e = ids[m], of the forward (b, onto the projection's result) and, with w's columns along n, of the backward pass
// (a, onto dx).
//
// base and out are the bytes: 8 per float32 element against 6 R flops (three terms of t).  A wave keeps the operand t
// of its 32 rows in registers (all ranks, three bfloat16 terms) and walks over n in strips of 64, loading base and the
// adapter's weights of the whole strip at once; there is no barrier and, forward, no LDS.  The output is computed
// transposed (MFMA rows are n), so a lane holds 4 consecutive n of one row and moves base and out in 16-byte pieces.
// A tile whose rows name several adapters is computed once per adapter, each storing its own rows; rows without an
// adapter are copied by the first.
#include <algorithm>

#include "lora_common.h"

namespace wq {

namespace {

using namespace lora;

constexpr int kStrip = 64;

// 4 consecutive elements at p (type ot) from index n on, those at D and beyond 0.  VEC: the 4 are aligned and inside.
__device__ __forceinline__ f32x4 load_out4(const uint8_t* p, int ot, int n, int D, bool vec) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (ot == X_F32) {
    if (vec) return *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < D) v[j] = reinterpret_cast<const float*>(p)[j];
    return v;
  }
  uint32_t h[4] = {0, 0, 0, 0};
  if (vec) {
    const u32x2 q = *reinterpret_cast<const u32x2*>(p);
    h[0] = q.x & 0xFFFFu; h[1] = q.x >> 16; h[2] = q.y & 0xFFFFu; h[3] = q.y >> 16;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < D) h[j] = reinterpret_cast<const uint16_t*>(p)[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = ot == X_BF16 ? bf16_bits_to_f32(h[j]) : (float)f16_from_bits((uint16_t)h[j]);
  return v;
}
__device__ __forceinline__ void store_out4(uint8_t* p, int ot, int n, int D, bool vec, f32x4 v) {
  if (ot == X_F32) {
    if (vec) {
      *reinterpret_cast<f32x4*>(p) = v;
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < D) reinterpret_cast<float*>(p)[j] = v[j];
    return;
  }
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float f = v[j];
    h[j] = ot == X_BF16 ? (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f) : (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f);
  }
  if (vec) {
    *reinterpret_cast<u32x2*>(p) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < D) reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)h[j];
}

template <int WT, bool TRANS, int NK>
__global__ void __launch_bounds__(256) lora_expand_kernel(int M, int D, int E, int R, int S, int strips, int nx,
                                                          const float* __restrict__ t, const uint8_t* __restrict__ w,
                                                          const float* __restrict__ scale, const int32_t* __restrict__ ids,
                                                          const uint8_t* base, uint8_t* out, int ot) {
  constexpr int NW = terms<WT>();
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int rt = (int)blockIdx.x / nx;
  const int m0 = rt * kRows;
  const int n_begin = (((int)blockIdx.x - rt * nx) * 4 + wave) * kStrip * strips, n_end = min(n_begin + kStrip * strips, D);
  const int es = ot == X_F32 ? 4 : 2;
  const int id = tile_id(ids, m0, M, E);
  uint32_t lead = tile_leaders(id);
  const bool aligned = (D & 3) == 0;

  // rows without an adapter: out = base
  const uint32_t bare = (uint32_t)__ballot(id < 0 && m0 + (lane & 31) < M);
  if (blockIdx.z == 0 && bare != 0 && base != out) {
    for (int n0 = n_begin; n0 < n_end; n0 += kStrip)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = 16 * i + l16, n = n0 + 16 * q + 4 * g;
          if (!(bare >> row & 1) || n >= n_end) continue;
          const size_t o = ((size_t)(m0 + row) * D + n) * es;
          const bool vec = aligned && n + 4 <= D;
          const f32x4 v = base ? load_out4(base + o, ot, n, D, vec) : f32x4{0.f, 0.f, 0.f, 0.f};
          store_out4(out + o, ot, n, D, vec, v);
        }
  }

  for (int z = 0; lead != 0; ++z, lead &= lead - 1) {
    if (z % (int)gridDim.z != (int)blockIdx.z) continue;
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctz(lead));
    const uint32_t mask = tile_mask(id, e);
    const uint8_t* we = w + (size_t)e * R * D * esize<WT>();
    const float f = scale[e];
    const bool on[2] = {(mask >> l16 & 1) != 0, (mask >> (16 + l16) & 1) != 0};
    // t of the two 16-row blocks: lane holds row l16 of the block, ranks 32 k + 8 g .. + 7
    bf16x8 tf[2][NK][3];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int r = 32 * k + 8 * g;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (on[i] && r < R) {
          const float* p = t + (size_t)(m0 + 16 * i + l16) * R + r;
          for (int s = 0; s < S; ++s, p += (size_t)M * R) {
            const f32x4 u0 = *reinterpret_cast<const f32x4*>(p), u1 = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] += u0[j];
              v[4 + j] += u1[j];
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= f;
        }
        split3<8>(v, tf[i][k]);
      }

    uint8_t* tile = lds + wave * NW * tr_plane<kStrip>();
    for (int n0 = n_begin; n0 < n_end; n0 += kStrip) {
      f32x4 y[4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = n0 + 16 * q + 4 * g;
          y[q][i] = f32x4{0.f, 0.f, 0.f, 0.f};
          if (base && on[i] && n < n_end)
            y[q][i] = load_out4(base + ((size_t)(m0 + 16 * i + l16) * D + n) * es, ot, n, D, aligned && n + 4 <= D);
        }
      f32x4 acc[4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[q][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        Raw<WT> raw[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (TRANS) {                       // rows r of D elements: chunk of the 32 x 64 tile
            const int c = lane + 64 * q, r = 32 * k + (c >> 3), n = n0 + 8 * (c & 7);
            if (r < R && n < D) raw_load<WT, true>(we + ((size_t)r * D + n) * esize<WT>(), raw[q]);
            else raw_zero(raw[q]);
          } else {
            const int r = 32 * k + 8 * g, n = n0 + 16 * q + l16;
            if (r < R && n < D) raw_load<WT, true>(we + ((size_t)n * R + r) * esize<WT>(), raw[q]);
            else raw_zero(raw[q]);
          }
        }
        if constexpr (TRANS) {
          wave_lds_fence();
#pragma unroll
          for (int q = 0; q < 4; ++q) tr_write<WT, kStrip>(tile, lane + 64 * q, raw[q]);
          wave_lds_fence();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          bf16x8 wf[NW];
          if constexpr (TRANS) tr_read<kStrip, NW>(tile, q, wf);
          else raw_terms<WT>(raw[q], wf);
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[q][i] = mfma_terms<NW, 3>(wf, tf[i][k], acc[q][i]);
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = n0 + 16 * q + 4 * g;
          if (!on[i] || n >= n_end) continue;
          store_out4(out + ((size_t)(m0 + 16 * i + l16) * D + n) * es, ot, n, D, aligned && n + 4 <= D, y[q][i] + acc[q][i]);
        }
    }
  }
}

template <int WT, bool TRANS, int NK>
hipError_t go(int M, int D, int E, int R, int S, const float* t, const void* w, const float* scale, const int32_t* ids,
              const void* base, void* out, int ot, hipStream_t st) {
  constexpr int lds = TRANS ? 4 * terms<WT>() * tr_plane<kStrip>() : 0;
  if (lds > 0 && !raise_lds_limit<lora_expand_kernel<WT, TRANS, NK>>()) return hipErrorInvalidValue;
  const int tiles = (M + kRows - 1) / kRows;
  // strips per wave: more while the launch keeps over 2048 workgroups (t is loaded once per wave)
  int strips = 1;
  while (strips < 4 && (int64_t)tiles * ((D + 8 * strips * kStrip - 1) / (8 * strips * kStrip)) > 2048) strips *= 2;
  const int nx = (D + 4 * strips * kStrip - 1) / (4 * strips * kStrip);
  const int dz = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(E, kRows), 4096 / ((int64_t)tiles * nx)));
  hipLaunchKernelGGL((lora_expand_kernel<WT, TRANS, NK>), dim3((unsigned)(tiles * nx), 1, dz), dim3(256), lds, st, M, D, E, R, S,
                     strips, nx, t, reinterpret_cast<const uint8_t*>(w), scale, ids, reinterpret_cast<const uint8_t*>(base),
                     reinterpret_cast<uint8_t*>(out), ot);
  return hipGetLastError();
}
template <int WT, bool TRANS, typename... A>
hipError_t by_rank(int M, int D, int E, int R, A... a) {
  if (R <= 32) return go<WT, TRANS, 1>(M, D, E, R, a...);
  if (R <= 64) return go<WT, TRANS, 2>(M, D, E, R, a...);
  if (R <= 128) return go<WT, TRANS, 4>(M, D, E, R, a...);
  return go<WT, TRANS, 8>(M, D, E, R, a...);
}
template <bool TRANS, typename... A>
hipError_t by_weight(XType wt, A... a) {
  if (wt == X_F32) return by_rank<X_F32, TRANS>(a...);
  if (wt == X_BF16) return by_rank<X_BF16, TRANS>(a...);
  return by_rank<X_F16, TRANS>(a...);
}

}  // namespace

hipError_t lora_expand(int M, int D, int E, int R, int S, const float* t, const void* w, XType wt, bool trans,
                       const float* scale, const int32_t* ids, const void* base, void* out, XType ot, hipStream_t st) {
  if (trans) return by_weight<true>(wt, M, D, E, R, S, t, w, scale, ids, base, out, (int)ot, st);
  return by_weight<false>(wt, M, D, E, R, S, t, w, scale, ids, base, out, (int)ot, st);
}

}  // namespace wq
