// Low-rank adapters, the contraction to the rank (gfx950): t[m,r] = sum_d x[m,d] w[e][r,d], e = ids[m], of the
// forward (x, a) and, with w's rows along the contraction, of the backward pass (dy, b).
//
// x is read once and dominates the bytes for long batches.  A workgroup takes 32 rows; its waves take blocks of 64 d in
// turn and add their 32 x R sums through LDS at the end, so nothing is shared and no barrier stands in the loop.  An MFMA
// operand wants a row per lane; loading it that way touches a cache line per lane (16 useful bytes each), which bounded
// an earlier form at 2 TB/s, so a wave loads whole lines, writes them to LDS of its own and reads the operands there;
// the next block's loads fly during this block's MFMAs.  A tile whose rows name several adapters is computed once per
// adapter, by blockIdx.z-th workgroups of their own (a row's operands enter only its own row of the product, and only
// the adapter's rows are loaded and written).  Where few tiles have a long contraction, it is split over up to 8
// workgroups and lora_terms_kernel adds their parts in order.  Shortest and mean of 20 calls: 4096 x 17408 float32, rank 16: 46
// and 48 us (6.0-6.2 TB/s, a part of it from the last-level cache); 4099 x 5120 bfloat16, rank 64: 18 and 20 us; 2047 x 17408
// bfloat16, rank 32: 21 and 24 us (3.0-3.3 TB/s).  Short ones are a launch's latency (5 us at 256 columns) and the few CUs that
// 32-row tiles occupy.
//
// Few rows (decode): one wave per row and rank, plain float32 products; see lora_shrink_rows_kernel.
#include <algorithm>

#include "lora_common.h"

namespace wq {

namespace {

using namespace lora;

constexpr int kParts = 8;            // most parts of the contraction

// A wave's LDS: 32 rows of x and, as rows (16 NR of them) or as a transposing tile, w; a row of 64 elements is padded by
// 16 bytes, which spreads the operand reads of 16 rows over all banks.
template <int T> constexpr int row_bytes() { return 64 * esize<T>() + 16; }
template <int XT, int WT, bool TRANS, int NR> constexpr int shrink_wave_lds() {
  return kRows * row_bytes<XT>() + (TRANS ? terms<WT>() * tr_plane<16 * NR>() : 16 * NR * row_bytes<WT>());
}
// Waves of a workgroup: 8 where two workgroups then share a CU's LDS or an operand is float32, else (16-bit operands of rank 64)
// as many as one workgroup's LDS holds.
template <int XT, int WT, bool TRANS, int NR> constexpr int shrink_waves() {
  constexpr int each = shrink_wave_lds<XT, WT, TRANS, NR>(), n = 160 * 1024 / each;
  constexpr int most = 16 * each <= 160 * 1024 || XT == X_F32 || WT == X_F32 ? 8 : 16;
  return n < most ? n : most;
}
template <int XT, int WT, bool TRANS, int NR> constexpr int shrink_lds() {
  constexpr int waves = shrink_waves<XT, WT, TRANS, NR>();
  constexpr int red = waves * kRows * 16 * NR * 4, stage = waves * shrink_wave_lds<XT, WT, TRANS, NR>();
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
__global__ void __launch_bounds__((64 * shrink_waves<XT, WT, TRANS, NR>()))
    lora_shrink_kernel(int M, int D, int E, int R, int S, int RC, const uint8_t* __restrict__ x, const uint8_t* __restrict__ w,
                       const float* __restrict__ scale, const int32_t* __restrict__ ids, uint16_t* __restrict__ t,
                       float* __restrict__ parts) {
  constexpr int kWaves = shrink_waves<XT, WT, TRANS, NR>();
  constexpr int C = 16 * NR, NX = terms<XT>(), NW = terms<WT>();
  constexpr int XP = 16 / esize<XT>(), WP = 16 / esize<WT>();       // elements of a 16-byte piece
  constexpr int XL = 64 / XP, WL = 64 / WP;                          // pieces of a row of 64
  constexpr int XN = kRows * XL / 64, WN = TRANS ? 1 : C * WL / 64;  // pieces per lane
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  // parts fastest: those of one part tend to one XCD, whose L2 then holds that part of w only (2047 rows of 17408, rank 32 on 5
  // adapters, 8 parts: 21 us instead of 26)
  const int tile = (int)blockIdx.x / (S * RC), sr = (int)blockIdx.x - tile * (S * RC);
  const int m0 = tile * kRows, s = sr % S, r0 = sr / S * C;
  const int id = tile_id(ids, m0, M, E);
  uint32_t lead = tile_leaders(id);
  const int nb = (D + 63) / 64, per = (nb + S - 1) / S;
  const int b0 = s * per, b1 = min(b0 + per, nb);
  uint8_t* xt = lds + wave * shrink_wave_lds<XT, WT, TRANS, NR>();
  uint8_t* wt = xt + kRows * row_bytes<XT>();
  for (int z = 0; lead != 0; ++z, lead &= lead - 1) {
    if (z % (int)gridDim.z != (int)blockIdx.z) continue;
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctz(lead));
    const uint32_t mask = tile_mask(id, e);
    const uint8_t* we = w + (size_t)e * R * D * esize<WT>();

    f32x4 acc[2][NR];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // a block as loaded: piece q of x covers row c / XL, elements XP (c % XL) .. of the block, c = lane + 64 q
    u32x4 xr[XN], wr[WN];
    Raw<WT> wtr[TRANS ? 2 : 1][NR];
    auto load = [&](int b) {
      const bool whole = 64 * b + 64 <= D;               // the same for all lanes: no branch between the loads
#pragma unroll
      for (int q = 0; q < XN; ++q) {
        const int c = lane + 64 * q, row = c / XL, d = 64 * b + XP * (c % XL);
        const uint8_t* p = x + ((size_t)(m0 + row) * D + d) * esize<XT>();
        const bool on = (mask >> row & 1) != 0;
        xr[q] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (TRANS) {                         // x = dy: D may be any number
          if (whole ? on : on && d + XP <= D) {
            if constexpr (XT == X_F32) xr[q] = *reinterpret_cast<const u32x4_a4*>(p);
            else xr[q] = *reinterpret_cast<const u32x4_a2*>(p);
          }
        } else {                                       // D is a multiple of 16
          if (on && d < D) xr[q] = *reinterpret_cast<const u32x4*>(p);
        }
      }
      if constexpr (TRANS) {
        if (!whole) {                                    // the contraction's end: pieces that D cuts
#pragma unroll
          for (int q = 0; q < XN; ++q) {
            const int c = lane + 64 * q, row = c / XL, d = 64 * b + XP * (c % XL);
            if (!(mask >> row & 1) || d >= D || d + XP <= D) continue;
            Raw<XT> part;
            raw_load_part<XT>(x + ((size_t)(m0 + row) * D + d) * esize<XT>(), D - d, part);
            xr[q] = part.v[0];
          }
        }
      }
      if constexpr (TRANS) {                           // rows d, R contiguous: chunk c of the 32 x C tile of step k
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            const int c = lane + 64 * j, dr = 64 * b + 32 * k + c / (C / 8), r = r0 + 8 * (c % (C / 8));
            if (dr < D && r < R) raw_load<WT, true>(we + ((size_t)dr * R + r) * esize<WT>(), wtr[k][j]);
            else raw_zero(wtr[k][j]);
          }
      } else {
#pragma unroll
        for (int q = 0; q < WN; ++q) {
          const int c = lane + 64 * q, r = r0 + c / WL, d = 64 * b + WP * (c % WL);
          wr[q] = r < R && d < D ? *reinterpret_cast<const u32x4*>(we + ((size_t)r * D + d) * esize<WT>()) : u32x4{0u, 0u, 0u, 0u};
        }
      }
    };
    auto lds_raw = [](const uint8_t* p, auto& r) {     // 8 elements of a row
      r.v[0] = *reinterpret_cast<const u32x4*>(p);
      if constexpr (sizeof(r) == 32) r.v[1] = *reinterpret_cast<const u32x4*>(p + 16);
    };
    int b = b0 + wave;
    if (b < b1) load(b);
    for (; b < b1; b += kWaves) {
      wave_lds_fence();                                // the previous block's reads
#pragma unroll
      for (int q = 0; q < XN; ++q) {
        const int c = lane + 64 * q;
        *reinterpret_cast<u32x4*>(xt + (c / XL) * row_bytes<XT>() + (c % XL) * 16) = xr[q];
      }
      if constexpr (!TRANS) {
#pragma unroll
        for (int q = 0; q < WN; ++q) {
          const int c = lane + 64 * q;
          *reinterpret_cast<u32x4*>(wt + (c / WL) * row_bytes<WT>() + (c % WL) * 16) = wr[q];
        }
      } else {
#pragma unroll
        for (int j = 0; j < NR; ++j) tr_write<WT, C>(wt, lane + 64 * j, wtr[0][j]);
      }
      wave_lds_fence();
      Raw<WT> second[NR];
      if constexpr (TRANS) {
#pragma unroll
        for (int j = 0; j < NR; ++j) second[j] = wtr[1][j];
      }
      if (b + kWaves < b1) load(b + kWaves);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if constexpr (TRANS) {
          if (k == 1) {                                // the tile holds one step of 32 d at a time
            wave_lds_fence();
#pragma unroll
            for (int j = 0; j < NR; ++j) tr_write<WT, C>(wt, lane + 64 * j, second[j]);
            wave_lds_fence();
          }
        }
        bf16x8 xf[2][NX];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          Raw<XT> r;
          lds_raw(xt + (16 * i + l16) * row_bytes<XT>() + (32 * k + 8 * g) * esize<XT>(), r);
          raw_terms<XT>(r, xf[i]);
        }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          bf16x8 wf[NW];
          if constexpr (TRANS) {
            tr_read<C, NW>(wt, j, wf);
          } else {
            Raw<WT> r;
            lds_raw(wt + (16 * j + l16) * row_bytes<WT>() + (32 * k + 8 * g) * esize<WT>(), r);
            raw_terms<WT>(r, wf);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[i][j] = mfma_terms<NX, NW>(xf[i], wf, acc[i][j]);
        }
      }
    }

    // sums of the waves in wave order; acc element q of lane: row 4 g + q of the block, column l16
    float* red = reinterpret_cast<float*>(lds);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NR; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) red[(wave * kRows + 16 * i + 4 * g + q) * C + 16 * j + l16] = acc[i][j][q];
    __syncthreads();
    const float f = scale[e];
    for (int o = threadIdx.x; o < kRows * C; o += 64 * kWaves) {
      const int row = o / C, r = r0 + o % C;
      if (!(mask >> row & 1) || r >= R) continue;
      float v = red[o];
#pragma unroll
      for (int q = 1; q < kWaves; ++q) v += red[q * kRows * C + o];
      const size_t at = (size_t)(m0 + row) * R + r, plane = (size_t)M * R;
      if (S > 1) parts[s * plane + at] = v;
      else put_terms(t + at, plane, v * f);
    }
    __syncthreads();
  }
}

// Few rows: one wave per row and rank (61 rows x 5120, rank 16: 4.8 us, a launch's latency and a row's).  A lane takes 8 consecutive d of every 512, so a wave reads whole lines of x and of
// the adapter's row, 4 steps in flight; the products are float32.
template <int XT, int WT>
__global__ void __launch_bounds__(256) lora_shrink_rows_kernel(int M, int D, int E, int R, const uint8_t* __restrict__ x,
                                                               const uint8_t* __restrict__ w, const float* __restrict__ scale,
                                                               const int32_t* __restrict__ ids, uint16_t* __restrict__ t) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = (int)blockIdx.x, r = (int)blockIdx.y * 4 + wave;     // R is a multiple of 8
  const int e = ids[m];
  if (e < 0 || e >= E) return;
  const uint8_t* xr = x + (size_t)m * D * esize<XT>();
  const uint8_t* wr = w + ((size_t)e * R + r) * D * esize<WT>();
  float acc = 0.f;
  for (int d0 = 8 * lane; d0 < D; d0 += 2048) {
    Raw<XT> a[4];
    Raw<WT> b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int d = d0 + 512 * q;
      raw_zero(a[q]);
      raw_zero(b[q]);
      if (d < D) {
        raw_load<XT, true>(xr + (size_t)d * esize<XT>(), a[q]);
        raw_load<WT, true>(wr + (size_t)d * esize<WT>(), b[q]);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float u[8], v[8];
      raw_f32<XT>(a[q], u);
      raw_f32<WT>(b[q], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc = fmaf(u[j], v[j], acc);
    }
  }
  acc = wave64_sum(acc);
  if (lane == 0) put_terms(t + (size_t)m * R + r, (size_t)M * R, acc * scale[e]);
}

// Few rows, w's rows along the contraction: one workgroup per row.  The ranks of one d lie next to each other; G lanes (a power of
// two covering R / 8) share a d, each holding the sums of its 8 ranks, so a wave reads w in whole lines; the lanes' and the 16
// waves' sums are added at the end, in a fixed order.
template <int XT, int WT, int G>
__global__ void __launch_bounds__(1024) lora_shrink_rows_t_kernel(int M, int D, int E, int R, const uint8_t* __restrict__ x,
                                                                  const uint8_t* __restrict__ w, const float* __restrict__ scale,
                                                                  const int32_t* __restrict__ ids, uint16_t* __restrict__ t) {
  constexpr int DPW = 64 / G, STEP = 16 * DPW;   // d of a wave's and of the workgroup's step
  __shared__ float sums[16][8 * G];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = (int)blockIdx.x;
  const int e = ids[m];
  if (e < 0 || e >= E) return;
  const int c = lane % G;
  const bool on = 8 * c < R;
  const uint8_t* xr = x + (size_t)m * D * esize<XT>();
  const uint8_t* we = w + ((size_t)e * D * R + 8 * c) * esize<WT>();
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int d0 = wave * DPW + lane / G; d0 < D; d0 += 4 * STEP) {
    Raw<WT> raw[4];
    float xv[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int d = d0 + q * STEP;
      raw_zero(raw[q]);
      xv[q] = 0.f;
      if (on && d < D) {
        raw_load<WT, true>(we + (size_t)d * R * esize<WT>(), raw[q]);
        xv[q] = XT == X_F32 ? reinterpret_cast<const float*>(xr)[d] : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(xr)[d]);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[8];
      raw_f32<WT>(raw[q], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = fmaf(xv[q], v[j], acc[j]);
    }
  }
#pragma unroll
  for (int off = 32; off >= G; off >>= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += __shfl_xor(acc[j], off, 64);
  if (lane < G) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[wave][8 * lane + j] = acc[j];
  }
  __syncthreads();
  const int r = threadIdx.x;
  if (r >= R) return;
  float v = sums[0][r];
#pragma unroll
  for (int q = 1; q < 16; ++q) v += sums[q][r];
  put_terms(t + (size_t)m * R + r, (size_t)M * R, v * scale[e]);
}

// Terms of the sums of S parts, in order: one thread per element.
__global__ void __launch_bounds__(256) lora_terms_kernel(int plane, int E, int R, int S, const float* __restrict__ parts,
                                                         const float* __restrict__ scale, const int32_t* __restrict__ ids,
                                                         uint16_t* __restrict__ t) {
  for (int i = blockIdx.x * 256 + threadIdx.x; i < plane; i += gridDim.x * 256) {
    const int e = ids[i / R];
    if (e < 0 || e >= E) continue;
    float p[kParts];                       // all loads in flight together
#pragma unroll
    for (int s = 0; s < kParts; ++s)
      if (s < S) p[s] = parts[s * plane + i];
    float v = p[0];
#pragma unroll
    for (int s = 1; s < kParts; ++s)
      if (s < S) v += p[s];
    put_terms(t + i, plane, v * scale[e]);
  }
}

// Parts of the contraction, at most 8, two workgroups per CU: where fewer than a workgroup per CU would read over 512 KB of x each,
// or much of x and w together.  512 KB of both with at most 32 workgroups (64 rows of 7007 bfloat16, rank 64: 15 us instead of 27;
// one row, rank 128, float32 w: 19 instead of 57), else 1.5 MB, below which the parts' own launch takes what they gain (2048 rows,
// rank 64, of 7007: float32 w 42 instead of 62, bfloat16 w 33 instead of 31).
int shrink_parts(int M, int D, int R, int es, int ws) {
  const int tiles = ((M + kRows - 1) / kRows) * ((R + 63) / 64);
  if (tiles == 0) return 1;                // no rows: the size queries and the weight gradients (zeros) still come here
  const int64_t xb = (int64_t)kRows * D * es, wb = (int64_t)std::min(R, 64) * D * ws;
  if (tiles >= 256 || (xb <= (512 << 10) && xb + wb <= (tiles <= 32 ? 512 << 10 : 1536 << 10))) return 1;
  const int s = std::min(kParts, 512 / tiles);
  if (s <= 1) return 1;
  const int nb = (D + 63) / 64, per = (nb + s - 1) / s;
  return (nb + per - 1) / per;             // no empty part
}

template <int XT, int WT, bool TRANS, int NR>
hipError_t go(int M, int D, int E, int R, int S, const void* x, const void* w, const float* scale, const int32_t* ids,
              uint16_t* t, float* parts, hipStream_t st) {
  if (!raise_lds_limit<lora_shrink_kernel<XT, WT, TRANS, NR>>()) return hipErrorInvalidValue;
  const int tiles = (M + kRows - 1) / kRows, RC = (R + 16 * NR - 1) / (16 * NR);
  // workgroups for further adapters of a tile, at least two; what they leave, each does in turn
  const int dz = std::min(std::min(E, kRows), std::max(2, 512 / std::max(1, tiles * S * RC)));
  hipLaunchKernelGGL((lora_shrink_kernel<XT, WT, TRANS, NR>), dim3(tiles * S * RC, 1, dz),
                     dim3(64 * shrink_waves<XT, WT, TRANS, NR>()), (shrink_lds<XT, WT, TRANS, NR>()), st, M, D, E, R, S, RC,
                     reinterpret_cast<const uint8_t*>(x), reinterpret_cast<const uint8_t*>(w), scale, ids, t, parts);
  return hipGetLastError();
}
template <int XT, int WT, bool TRANS, typename... A>
hipError_t by_rank(int M, int D, int E, int R, A... a) {
  if (R <= 16) return go<XT, WT, TRANS, 1>(M, D, E, R, a...);
  if (R <= 32) return go<XT, WT, TRANS, 2>(M, D, E, R, a...);
  return go<XT, WT, TRANS, 4>(M, D, E, R, a...);
}
template <int XT, int WT>
hipError_t go_rows(int M, int D, int E, int R, const void* x, const void* w, const float* scale, const int32_t* ids, uint16_t* t,
                   hipStream_t st) {
  hipLaunchKernelGGL((lora_shrink_rows_kernel<XT, WT>), dim3(M, R / 4), dim3(256), 0, st, M, D, E, R,
                     reinterpret_cast<const uint8_t*>(x), reinterpret_cast<const uint8_t*>(w), scale, ids, t);
  return hipGetLastError();
}
template <int XT, typename... A>
hipError_t rows_by_weight(XType wt, A... a) {
  if (wt == X_F32) return go_rows<XT, X_F32>(a...);
  if (wt == X_BF16) return go_rows<XT, X_BF16>(a...);
  return go_rows<XT, X_F16>(a...);
}
template <int XT, int WT, int G>
hipError_t go_rows_t(int M, int D, int E, int R, const void* x, const void* w, const float* scale, const int32_t* ids,
                     uint16_t* t, hipStream_t st) {
  hipLaunchKernelGGL((lora_shrink_rows_t_kernel<XT, WT, G>), dim3(M), dim3(1024), 0, st, M, D, E, R,
                     reinterpret_cast<const uint8_t*>(x), reinterpret_cast<const uint8_t*>(w), scale, ids, t);
  return hipGetLastError();
}
template <int XT, int WT, typename... A>
hipError_t rows_t_by_rank(int M, int D, int E, int R, A... a) {
  if (R <= 8) return go_rows_t<XT, WT, 1>(M, D, E, R, a...);
  if (R <= 16) return go_rows_t<XT, WT, 2>(M, D, E, R, a...);
  if (R <= 32) return go_rows_t<XT, WT, 4>(M, D, E, R, a...);
  if (R <= 64) return go_rows_t<XT, WT, 8>(M, D, E, R, a...);
  if (R <= 128) return go_rows_t<XT, WT, 16>(M, D, E, R, a...);
  return go_rows_t<XT, WT, 32>(M, D, E, R, a...);
}
template <int XT, typename... A>
hipError_t rows_t_by_weight(XType wt, A... a) {
  if (wt == X_F32) return rows_t_by_rank<XT, X_F32>(a...);
  if (wt == X_BF16) return rows_t_by_rank<XT, X_BF16>(a...);
  return rows_t_by_rank<XT, X_F16>(a...);
}
template <int XT, bool TRANS, typename... A>
hipError_t by_weight(XType wt, A... a) {
  if (wt == X_F32) return by_rank<XT, X_F32, TRANS>(a...);
  if (wt == X_BF16) return by_rank<XT, X_BF16, TRANS>(a...);
  return by_rank<XT, X_F16, TRANS>(a...);
}

}  // namespace

size_t lora_shrink_bytes(int M, int D, int R, XType xt) {
  const int s = shrink_parts(M, D, R, xt == X_F32 ? 4 : 2, 4);      // of any weights
  return s > 1 ? (size_t)s * M * R * 4 : 0;
}

hipError_t lora_shrink(bool few, int M, int D, int E, int R, const void* x, XType xt, const void* w, XType wt, bool trans,
                       const float* scale, const int32_t* ids, uint16_t* t, float* parts, hipStream_t st) {
  // transposed: a workgroup reads a whole adapter matrix, at some 150 GB/s
  if (few && trans && (int64_t)D * R * (wt == X_F32 ? 4 : 2) <= (512 << 10)) {
    if (xt == X_F32) return rows_t_by_weight<X_F32>(wt, M, D, E, R, x, w, scale, ids, t, st);
    return rows_t_by_weight<X_BF16>(wt, M, D, E, R, x, w, scale, ids, t, st);
  }
  if (few && !trans) {
    if (xt == X_F32) return rows_by_weight<X_F32>(wt, M, D, E, R, x, w, scale, ids, t, st);
    if (xt == X_BF16) return rows_by_weight<X_BF16>(wt, M, D, E, R, x, w, scale, ids, t, st);
    return rows_by_weight<X_F16>(wt, M, D, E, R, x, w, scale, ids, t, st);
  }
  const int S = shrink_parts(M, D, R, xt == X_F32 ? 4 : 2, wt == X_F32 ? 4 : 2);
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
  const int plane = M * R;                 // parts are for less than 256 tiles of 32 rows
  hipLaunchKernelGGL(lora_terms_kernel, dim3((unsigned)std::min((plane + 255) / 256, 4096)), dim3(256), 0, st, plane, E,
                     R, S, parts, scale, ids, t);
  return hipGetLastError();
}

}  // namespace wq
