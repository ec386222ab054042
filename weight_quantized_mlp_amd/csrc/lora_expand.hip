// Low-rank adapters, the product back from the rank (gfx950): out[m,n] = base[m,n] + sum_r t[m,r] w[e][n,r],
// e = ids[m], t scaled already, of the forward (b, onto the projection's result) and, with w's columns along n, of the backward pass
// (a, onto dx).
//
// base and out are the bytes: 8 per float32 element against 6 R flops (three terms of t).  A wave keeps the operand t
// of its 32 rows in registers (all ranks, three bfloat16 terms) and walks over n in strips of 64, loading base and the
// adapter's weights of the whole strip at once; there is no barrier and, forward, no LDS.  The output is computed
// transposed (MFMA rows are n), so a lane holds 4 or 8 consecutive n of one row and moves base and out in 16-byte pieces.
// A tile whose rows name several adapters is computed once per adapter, each storing its own rows; rows without an
// adapter are copied by the first.
#include <algorithm>

#include "lora_common.h"

namespace wq {

namespace {

using namespace lora;

// Columns a wave takes at a time, by rank steps: half as many where the operand t takes more registers.
template <int NK> constexpr int kStrip = NK == 1 ? 64 : 32;

// Output pieces.  float32: 4 consecutive elements from index n on (those at D and beyond read as 0 and are not written);
// VEC: the 4 are aligned and inside.
__device__ __forceinline__ f32x4 load_out4(const uint8_t* p, int n, int D, bool vec) {
  if (vec) return *reinterpret_cast<const f32x4*>(p);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < D) v[j] = reinterpret_cast<const float*>(p)[j];
  return v;
}
__device__ __forceinline__ void store_out4(uint8_t* p, int n, int D, bool vec, f32x4 v) {
  if (vec) {
    *reinterpret_cast<f32x4*>(p) = v;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < D) reinterpret_cast<float*>(p)[j] = v[j];
}
// 16-bit outputs: 8 consecutive elements, always aligned and inside (D is a multiple of 16 there).
__device__ __forceinline__ void load_out8(const uint8_t* p, int ot, f32x4& a, f32x4& b) {
  const u32x4 q = *reinterpret_cast<const u32x4*>(p);
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t d = q[j];
    v[2 * j] = ot == X_BF16 ? bf16_bits_to_f32(d & 0xFFFFu) : (float)f16_from_bits((uint16_t)d);
    v[2 * j + 1] = ot == X_BF16 ? bf16_bits_to_f32(d >> 16) : (float)f16_from_bits((uint16_t)(d >> 16));
  }
  a = f32x4{v[0], v[1], v[2], v[3]};
  b = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store_out8(uint8_t* p, int ot, f32x4 a, f32x4 b) {
  uint32_t h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = j < 4 ? a[j & 3] : b[j & 3];
    h[j] = ot == X_BF16 ? (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f) : (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f);
  }
  *reinterpret_cast<u32x4*>(p) = u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
}

// NK: rank steps of 32.  W16: out has 16-bit elements, and a lane then holds 8 consecutive n (two MFMA row blocks
// interleaved in fours), so that its piece of a row is 16 bytes there too.
template <int WT, bool TRANS, int NK, bool W16>
__global__ void __launch_bounds__(256) lora_expand_kernel(int M, int D, int E, int R, int strips, int nx,
                                                          const uint16_t* __restrict__ t, const uint8_t* __restrict__ w,
                                                          const int32_t* __restrict__ ids, const uint8_t* base, uint8_t* out,
                                                          int ot) {
  constexpr int NW = terms<WT>();
  constexpr int ES = W16 ? 2 : 4;
  constexpr int Q = kStrip<NK> / 16;           // MFMA row blocks of a strip
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int rt = (int)blockIdx.x / nx;
  const int m0 = rt * kRows;
  const int n_begin = (((int)blockIdx.x - rt * nx) * 4 + wave) * kStrip<NK> * strips;
  const int n_end = min(n_begin + kStrip<NK> * strips, D);
  const int id = tile_id(ids, m0, M, E);
  uint32_t lead = tile_leaders(id);
  const bool aligned = (D & 3) == 0;
  // first n of the 4 that MFMA row block q leaves in this lane (accumulator rows 4 g .. + 3)
  auto n_of = [&](int q) { return W16 ? 32 * (q >> 1) + 8 * g + 4 * (q & 1) : 16 * q + 4 * g; };

  // the strip's pieces of the rows whose bit in `rows` is set
  auto load_rows = [&](uint32_t rows, int n0, f32x4 (&y)[Q][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 16 * i + l16;
      const bool on = base != nullptr && (rows >> row & 1) != 0;
      const uint8_t* p = base + (size_t)(m0 + row) * D * ES;
#pragma unroll
      for (int q = 0; q < Q; q += W16 ? 2 : 1) {
        const int n = n0 + n_of(q);
        y[q][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (W16) {
          y[q + 1][i] = f32x4{0.f, 0.f, 0.f, 0.f};
          if (on && n < n_end) load_out8(p + (size_t)n * ES, ot, y[q][i], y[q + 1][i]);
        } else {
          if (on && n < n_end) y[q][i] = load_out4(p + (size_t)n * ES, n, D, aligned && n + 4 <= D);
        }
      }
    }
  };
  auto store_rows = [&](uint32_t rows, int n0, const f32x4 (&y)[Q][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 16 * i + l16;
      const bool on = (rows >> row & 1) != 0;
      uint8_t* p = out + (size_t)(m0 + row) * D * ES;
#pragma unroll
      for (int q = 0; q < Q; q += W16 ? 2 : 1) {
        const int n = n0 + n_of(q);
        if (!on || n >= n_end) continue;
        if constexpr (W16) store_out8(p + (size_t)n * ES, ot, y[q][i], y[q + 1][i]);
        else store_out4(p + (size_t)n * ES, n, D, aligned && n + 4 <= D, y[q][i]);
      }
    }
  };

  // rows without an adapter: out = base
  const uint32_t bare = (uint32_t)__ballot(id < 0 && m0 + (lane & 31) < M);
  if (blockIdx.z == 0 && bare != 0 && base != out) {
    for (int n0 = n_begin; n0 < n_end; n0 += kStrip<NK>) {
      f32x4 y[Q][2];
      load_rows(bare, n0, y);
      store_rows(bare, n0, y);
    }
  }

  uint8_t* tile = lds + wave * NW * tr_plane<kStrip<NK>>();
  for (int z = 0; lead != 0; ++z, lead &= lead - 1) {
    if (z % (int)gridDim.z != (int)blockIdx.z) continue;
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctz(lead));
    const uint32_t mask = tile_mask(id, e);
    const uint8_t* we = w + (size_t)e * R * D * esize<WT>();
    const bool on[2] = {(mask >> l16 & 1) != 0, (mask >> (16 + l16) & 1) != 0};
    f32x4 y[Q][2];
    Raw<WT> raw[Q];
    auto load_w = [&](int n0, int k) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if constexpr (TRANS) {                         // rows r of D elements: chunk of the 32 x strip tile
          constexpr int CW = kStrip<NK> / 8;
          const int c = lane + 64 * q, r = 32 * k + c / CW, n = n0 + 8 * (c % CW);
          if (r < R && n < D) raw_load<WT, true>(we + ((size_t)r * D + n) * esize<WT>(), raw[q]);
          else raw_zero(raw[q]);
        } else {                                       // operand row l16 of block q is n_of's n
          const int r = 32 * k + 8 * g;
          const int n = n0 + (W16 ? 32 * (q >> 1) + 8 * (l16 >> 2) + 4 * (q & 1) + (l16 & 3) : 16 * q + l16);
          if (r < R && n < D) raw_load<WT, true>(we + ((size_t)n * R + r) * esize<WT>(), raw[q]);
          else raw_zero(raw[q]);
        }
      }
    };
    if (n_begin < n_end) {
      load_w(n_begin, 0);
      load_rows(mask, n_begin, y);
    }
    // t of the two 16-row blocks: lane holds row l16 of the block, ranks 32 k + 8 g .. + 7
    bf16x8 tf[2][NK][3];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int r = 32 * k + 8 * g;
        const uint16_t* p = t + (size_t)(m0 + 16 * i + l16) * R + r;
#pragma unroll
        for (int q = 0; q < 3; ++q)
          tf[i][k][q] = __builtin_bit_cast(bf16x8, on[i] && r < R ? *reinterpret_cast<const u32x4*>(p + q * (size_t)M * R)
                                                                 : u32x4{0u, 0u, 0u, 0u});
      }

    for (int n0 = n_begin; n0 < n_end; n0 += kStrip<NK>) {
      f32x4 acc[Q][2];
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[q][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        bf16x8 wf[Q][NW];
        if constexpr (TRANS) {
          wave_lds_fence();
#pragma unroll
          for (int q = 0; q < Q; ++q) tr_write<WT, kStrip<NK>>(tile, lane + 64 * q, raw[q]);
          wave_lds_fence();
        } else {
#pragma unroll
          for (int q = 0; q < Q; ++q) raw_terms<WT>(raw[q], wf[q]);
        }
        // the next weights (this strip's next rank step, or the next strip's first) fly during the MFMAs
        if (k + 1 < NK) load_w(n0, k + 1);
        else if (n0 + kStrip<NK> < n_end) load_w(n0 + kStrip<NK>, 0);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          if constexpr (TRANS) tr_read<kStrip<NK>, NW, W16>(tile, q, wf[q]);
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[q][i] = mfma_terms<NW, 3>(wf[q], tf[i][k], acc[q][i]);
        }
      }
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[q][i] += y[q][i];
      if (n0 + kStrip<NK> < n_end) load_rows(mask, n0 + kStrip<NK>, y);
      store_rows(mask, n0, acc);
    }
  }
}

template <int WT, bool TRANS, int NK, bool W16>
hipError_t go(int M, int D, int E, int R, const uint16_t* t, const void* w, const int32_t* ids, const void* base, void* out,
              int ot, hipStream_t st) {
  constexpr int lds = TRANS ? 4 * terms<WT>() * tr_plane<kStrip<NK>>() : 0;
  if (lds > 0 && !raise_lds_limit<lora_expand_kernel<WT, TRANS, NK, W16>>()) return hipErrorInvalidValue;
  const int tiles = (M + kRows - 1) / kRows;
  // strips per wave: more while the launch keeps over 2048 workgroups (t is loaded once per wave)
  constexpr int kGroup = 4 * kStrip<NK>;
  int strips = 1;
  while (strips < 256 / kStrip<NK> && (int64_t)tiles * ((D + 2 * strips * kGroup - 1) / (2 * strips * kGroup)) > 2048) strips *= 2;
  const int nx = (D + strips * kGroup - 1) / (strips * kGroup);
  const int dz = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(E, kRows), 4096 / ((int64_t)tiles * nx)));
  hipLaunchKernelGGL((lora_expand_kernel<WT, TRANS, NK, W16>), dim3((unsigned)(tiles * nx), 1, dz), dim3(256), lds, st, M, D, E, R,
                     strips, nx, t, reinterpret_cast<const uint8_t*>(w), ids, reinterpret_cast<const uint8_t*>(base),
                     reinterpret_cast<uint8_t*>(out), ot);
  return hipGetLastError();
}
template <int WT, bool TRANS, bool W16, typename... A>
hipError_t by_rank(int M, int D, int E, int R, A... a) {
  if (R <= 32) return go<WT, TRANS, 1, W16>(M, D, E, R, a...);
  if (R <= 64) return go<WT, TRANS, 2, W16>(M, D, E, R, a...);
  if (R <= 128) return go<WT, TRANS, 4, W16>(M, D, E, R, a...);
  return go<WT, TRANS, 8, W16>(M, D, E, R, a...);
}
template <bool TRANS, bool W16, typename... A>
hipError_t by_weight(XType wt, A... a) {
  if (wt == X_F32) return by_rank<X_F32, TRANS, W16>(a...);
  if (wt == X_BF16) return by_rank<X_BF16, TRANS, W16>(a...);
  return by_rank<X_F16, TRANS, W16>(a...);
}

}  // namespace

// Forward (not trans) the output is float32, backward any type.
hipError_t lora_expand(int M, int D, int E, int R, const uint16_t* t, const void* w, XType wt, bool trans,
                       const int32_t* ids, const void* base, void* out, XType ot, hipStream_t st) {
  if (!trans) return ot == X_F32 ? by_weight<false, false>(wt, M, D, E, R, t, w, ids, base, out, (int)ot, st) : hipErrorInvalidValue;
  if (ot == X_F32) return by_weight<true, false>(wt, M, D, E, R, t, w, ids, base, out, (int)ot, st);
  return by_weight<true, true>(wt, M, D, E, R, t, w, ids, base, out, (int)ot, st);
}

}  // namespace wq
