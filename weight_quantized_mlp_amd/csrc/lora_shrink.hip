// Low-rank adapters, the contraction to the rank (gfx950): t[m,r] = sum_d x[m,d] w[e][r,d], e = ids[m], of the
// forward (x, a) and, with w's rows along the contraction, of the backward pass (dy, b).
//
// x is read once and dominates the bytes for long batches; for a few tokens the used adapters do.  A workgroup takes
// 32 rows; its waves take blocks of 64 d in turn and add their 32 x R sums through LDS at the end, so nothing is
// shared and no barrier stands in the loop.  Operands of 16 bits leave room for 16 waves, which cover the latency by
// their number; wider ones run 8 waves that load their next block during the MFMAs of this one.  A tile whose rows
// name several adapters is computed once per adapter, by blockIdx.z-th workgroups of their own (a row's operands
// enter only its own row of the product, and only the adapter's rows are loaded and written).  Where few tiles have a
// long contraction, it is split over up to 8 workgroups and lora_terms_kernel adds their parts in order.
#include <algorithm>

#include "lora_common.h"

namespace wq {

namespace {

using namespace lora;

// Waves of a workgroup: 16 where a wave's registers (at most 128 then) hold a block and its sums.
template <int XT, int WT, int NR> constexpr int shrink_waves() {
  return (XT != X_F32 && WT != X_F32) || (XT == X_F32 && WT != X_F32 && NR <= 2) ? 16 : 8;
}
constexpr int kRed = 8;              // waves whose sums LDS holds at once

template <int XT, int WT, bool TRANS, int NR> constexpr int shrink_lds() {
  const int red = kRed * kRows * 16 * NR * 4;
  const int stage = TRANS ? shrink_waves<XT, WT, NR>() * terms<WT>() * tr_plane<16 * NR>() : 0;
  return red > stage ? red : stage;
}

// The three bfloat16 terms of v, one per plane.
__device__ __forceinline__ void put_terms(uint16_t* t, size_t plane, float v) {
  __bf16 h[3][1];
  split3<1>(&v, h);
#pragma unroll
  for (int i = 0; i < 3; ++i) t[i * plane] = __builtin_bit_cast(uint16_t, h[i][0]);
}

template <int XT, int WT, bool TRANS, int NR>
__global__ void __launch_bounds__((64 * shrink_waves<XT, WT, NR>()))
    lora_shrink_kernel(int M, int D, int E, int R, int S, int RC, const uint8_t* __restrict__ x, const uint8_t* __restrict__ w,
                       const float* __restrict__ scale, const int32_t* __restrict__ ids, uint16_t* __restrict__ t,
                       float* __restrict__ parts) {
  constexpr int kWaves = shrink_waves<XT, WT, NR>();
  constexpr int C = 16 * NR, NX = terms<XT>(), NW = terms<WT>();
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int m0 = (int)blockIdx.x * kRows;
  const int s = (int)blockIdx.y / RC, r0 = ((int)blockIdx.y - s * RC) * C;
  const int id = tile_id(ids, m0, M, E);
  uint32_t lead = tile_leaders(id);
  const int nb = (D + 63) / 64, per = (nb + S - 1) / S;
  const int b0 = s * per, b1 = min(b0 + per, nb);
  for (int z = 0; lead != 0; ++z, lead &= lead - 1) {
    if (z % (int)gridDim.z != (int)blockIdx.z) continue;
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctz(lead));
    const uint32_t mask = tile_mask(id, e);
    const uint8_t* we = w + (size_t)e * R * D * esize<WT>();
    // rows of the two 16-row blocks that this lane loads
    const bool on[2] = {(mask >> l16 & 1) != 0, (mask >> (16 + l16) & 1) != 0};
    const uint8_t* xr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) xr[i] = x + (size_t)(m0 + 16 * i + l16) * D * esize<XT>();

    f32x4 acc[2][NR];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // one block: 64 d as two MFMA steps of 32
    struct Block {
      Raw<XT> x[2][2];
      Raw<WT> w[2][TRANS ? (C + 15) / 16 : NR];
    };
    auto load = [&](int b, Block& k) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int d = 64 * b + 32 * q + 8 * g;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (TRANS) {                       // x = dy: D may be any number
            if (on[i] && d + 8 <= D) raw_load<XT, false>(xr[i] + (size_t)d * esize<XT>(), k.x[q][i]);
            else raw_load_part<XT>(xr[i] + (size_t)d * esize<XT>(), on[i] ? D - d : 0, k.x[q][i]);
          } else {                                     // D is a multiple of 16
            if (on[i] && d < D) raw_load<XT, true>(xr[i] + (size_t)d * esize<XT>(), k.x[q][i]);
            else raw_zero(k.x[q][i]);
          }
        }
        if constexpr (TRANS) {                         // rows d, R contiguous: chunk c of the 32 x C tile
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            const int c = lane + 64 * j, dr = 64 * b + 32 * q + c / (C / 8), r = r0 + 8 * (c % (C / 8));
            if (dr < D && r < R) raw_load<WT, true>(we + ((size_t)dr * R + r) * esize<WT>(), k.w[q][j]);
            else raw_zero(k.w[q][j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            const int r = r0 + 16 * j + l16;
            if (r < R && d < D) raw_load<WT, true>(we + ((size_t)r * D + d) * esize<WT>(), k.w[q][j]);
            else raw_zero(k.w[q][j]);
          }
        }
      }
    };
    uint8_t* tile = lds + wave * NW * tr_plane<C>();
    auto compute = [&](const Block& k) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        bf16x8 xf[2][NX];
#pragma unroll
        for (int i = 0; i < 2; ++i) raw_terms<XT>(k.x[q][i], xf[i]);
        if constexpr (TRANS) {
          wave_lds_fence();                            // the previous step's reads
#pragma unroll
          for (int j = 0; j < NR; ++j) tr_write<WT, C>(tile, lane + 64 * j, k.w[q][j]);
          wave_lds_fence();
        }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          bf16x8 wf[NW];
          if constexpr (TRANS) tr_read<C, NW>(tile, j, wf);
          else raw_terms<WT>(k.w[q][j], wf);
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[i][j] = mfma_terms<NX, NW>(xf[i], wf, acc[i][j]);
        }
      }
    };
    if constexpr (kWaves == 16) {
      Block k;
      for (int b = b0 + wave; b < b1; b += kWaves) {
        load(b, k);
        compute(k);
      }
    } else {
      Block k0, k1;
      int b = b0 + wave;
      if (b < b1) load(b, k0);
      while (b < b1) {
        const bool more = b + kWaves < b1;
        if (more) load(b + kWaves, k1);
        compute(k0);
        if (!more) break;
        b += kWaves;
        if (b + kWaves < b1) load(b + kWaves, k0);
        compute(k1);
        b += kWaves;
      }
    }

    // sums of the waves in a fixed order; acc element q of lane: row 4 g + q of the block, column l16
    float* red = reinterpret_cast<float*>(lds);
    auto each = [&](auto f) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) f(i, j, q, ((wave % kRed) * kRows + 16 * i + 4 * g + q) * C + 16 * j + l16);
    };
    __syncthreads();
    if constexpr (kWaves == 16) {
      if (wave >= kRed) each([&](int i, int j, int q, int at) { red[at] = acc[i][j][q]; });
      __syncthreads();
      if (wave < kRed) each([&](int i, int j, int q, int at) { red[at] = acc[i][j][q] + red[at]; });
    } else {
      each([&](int i, int j, int q, int at) { red[at] = acc[i][j][q]; });
    }
    __syncthreads();
    const float f = scale[e];
    for (int o = threadIdx.x; o < kRows * C; o += 64 * kWaves) {
      const int row = o / C, r = r0 + o % C;
      if (!(mask >> row & 1) || r >= R) continue;
      float v = red[o];
#pragma unroll
      for (int q = 1; q < kRed; ++q) v += red[q * kRows * C + o];
      const size_t at = (size_t)(m0 + row) * R + r, plane = (size_t)M * R;
      if (S > 1) parts[s * plane + at] = v;
      else put_terms(t + at, plane, v * f);
    }
    __syncthreads();
  }
}

// Terms of the sums of S parts, in order: one thread per element.
__global__ void __launch_bounds__(256) lora_terms_kernel(int64_t plane, int E, int R, int S, const float* __restrict__ parts,
                                                         const float* __restrict__ scale, const int32_t* __restrict__ ids,
                                                         uint16_t* __restrict__ t) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < plane; i += (int64_t)gridDim.x * 256) {
    const int e = ids[i / R];
    if (e < 0 || e >= E) continue;
    float v = parts[i];
    for (int s = 1; s < S; ++s) v += parts[s * plane + i];
    put_terms(t + i, plane, v * scale[e]);
  }
}

// Parts of the contraction: where fewer than a workgroup per CU would read over 512 KB of x each, as many as bring that
// to 256 KB, at most 8 and two workgroups per CU.
int shrink_parts(int M, int D, int R, int es) {
  const int tiles = ((M + kRows - 1) / kRows) * ((R + 63) / 64);
  const int64_t bytes = (int64_t)kRows * D * es;
  if (tiles >= 256 || bytes <= (512 << 10)) return 1;
  const int s = (int)std::min<int64_t>(std::min(8, 512 / tiles), (bytes + (256 << 10) - 1) / (256 << 10));
  if (s <= 1) return 1;
  const int nb = (D + 63) / 64, per = (nb + s - 1) / s;
  return (nb + per - 1) / per;             // no empty part
}

template <int XT, int WT, bool TRANS, int NR>
hipError_t go(int M, int D, int E, int R, int S, const void* x, const void* w, const float* scale, const int32_t* ids,
              uint16_t* t, float* parts, hipStream_t st) {
  if (!raise_lds_limit<lora_shrink_kernel<XT, WT, TRANS, NR>>()) return hipErrorInvalidValue;
  const int tiles = (M + kRows - 1) / kRows, RC = (R + 16 * NR - 1) / (16 * NR);
  // workgroups for further adapters of a tile: up to one per possible adapter while the launch stays small
  const int dz = std::max(1, std::min(std::min(E, kRows), 2048 / std::max(1, tiles * S * RC)));
  hipLaunchKernelGGL((lora_shrink_kernel<XT, WT, TRANS, NR>), dim3(tiles, S * RC, dz),
                     dim3(64 * shrink_waves<XT, WT, NR>()), (shrink_lds<XT, WT, TRANS, NR>()), st, M, D, E, R, S, RC,
                     reinterpret_cast<const uint8_t*>(x), reinterpret_cast<const uint8_t*>(w), scale, ids, t, parts);
  return hipGetLastError();
}
template <int XT, int WT, bool TRANS, typename... A>
hipError_t by_rank(int M, int D, int E, int R, A... a) {
  if (R <= 16) return go<XT, WT, TRANS, 1>(M, D, E, R, a...);
  if (R <= 32) return go<XT, WT, TRANS, 2>(M, D, E, R, a...);
  return go<XT, WT, TRANS, 4>(M, D, E, R, a...);
}
template <int XT, bool TRANS, typename... A>
hipError_t by_weight(XType wt, A... a) {
  if (wt == X_F32) return by_rank<XT, X_F32, TRANS>(a...);
  if (wt == X_BF16) return by_rank<XT, X_BF16, TRANS>(a...);
  return by_rank<XT, X_F16, TRANS>(a...);
}

}  // namespace

size_t lora_shrink_bytes(int M, int D, int R, XType xt) {
  const int s = shrink_parts(M, D, R, xt == X_F32 ? 4 : 2);
  return s > 1 ? (size_t)s * M * R * 4 : 0;
}

hipError_t lora_shrink(int M, int D, int E, int R, const void* x, XType xt, const void* w, XType wt, bool trans,
                       const float* scale, const int32_t* ids, uint16_t* t, float* parts, hipStream_t st) {
  const int S = shrink_parts(M, D, R, xt == X_F32 ? 4 : 2);
  hipError_t err;
  if (trans) {
    err = xt == X_F32 ? by_weight<X_F32, true>(wt, M, D, E, R, S, x, w, scale, ids, t, parts, st)
                      : by_weight<X_BF16, true>(wt, M, D, E, R, S, x, w, scale, ids, t, parts, st);
  } else {
    err = xt == X_F32    ? by_weight<X_F32, false>(wt, M, D, E, R, S, x, w, scale, ids, t, parts, st)
          : xt == X_BF16 ? by_weight<X_BF16, false>(wt, M, D, E, R, S, x, w, scale, ids, t, parts, st)
                         : by_weight<X_F16, false>(wt, M, D, E, R, S, x, w, scale, ids, t, parts, st);
  }
  if (err != hipSuccess || S == 1) return err;
  const int64_t plane = (int64_t)M * R;
  hipLaunchKernelGGL(lora_terms_kernel, dim3((unsigned)std::min<int64_t>((plane + 255) / 256, 4096)), dim3(256), 0, st, plane, E,
                     R, S, parts, scale, ids, t);
  return hipGetLastError();
}

}  // namespace wq
