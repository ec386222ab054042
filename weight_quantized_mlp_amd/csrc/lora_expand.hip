// Low-rank adapters, the product back from the rank (gfx950): out[m,n] = base[m,n] + sum_r t[m,r] w[e][n,r],
// e = ids[m], t scaled already, of the forward (b, onto the projection's result) and, with w's columns along n, of the backward pass
// (a, onto dx).
//
// base and out are the bytes: 8 per float32 element against 6 R flops (three terms of t).  A wave keeps the operand t
// of its 32 rows in registers (all ranks, three bfloat16 terms) and walks over n in strips, the weights and base of the
// next strip in flight during this strip's MFMAs; there is no barrier.  The sums leave the MFMAs a row per lane; adding
// and storing them that way would touch a cache line per lane, so they pass through LDS of the wave's own and meet base
// in whole lines (16 lanes on 256 consecutive bytes of a row).  A tile whose rows name several adapters is computed once
// per adapter, each storing its own rows; rows without an adapter are copied by the first.  Shortest and mean of 20 calls:
// 4099 rows x 17408, rank 64: 129 and 137 us (571 MB, 4.2-4.4 TB/s; with the products taken out 113); 2047 rows x 17408 bfloat16
// (dx), rank 32: 41 and 44 us.
//
// Few rows (decode): see lora_expand_rows_kernel.
#include <algorithm>

#include "../../include/wqmlp_adapters.h"
#include "lora_common.h"

namespace wq {

namespace {

using namespace lora;

// Columns a wave takes at a time, by rank steps: half as many where the operand t takes more registers.
template <int NK> constexpr int kStrip = NK == 1 ? 64 : 32;

// 16 bytes of a row of the output: 4 float32 (rows of any length: element-aligned) or 8 16-bit elements (rows of a multiple of
// 16) from n on; elements at D and beyond read as 0 and are not written.  Both streams pass the caches once, and say so (ONCE):
// the adapters' weights, which every row tile reads again, stay (4099 rows x 17408: 153 us without, 138 with it, when it was added).  See
// expand_once for rows that end inside a line.
template <bool ONCE, typename V>
__device__ __forceinline__ V load_as(const uint8_t* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
  else return *reinterpret_cast<const V*>(p);
}
template <bool ONCE, typename V>
__device__ __forceinline__ void store_as(uint8_t* p, V v) {
  if constexpr (ONCE) __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
  else *reinterpret_cast<V*>(p) = v;
}
template <bool W16, bool ONCE>
__device__ __forceinline__ u32x4 load_piece(const uint8_t* p, int n, int D) {
  if (W16) return load_as<ONCE, u32x4>(p);
  if (n + 4 <= D) return load_as<ONCE, u32x4_a4>(p);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (n + j < D) v[j] = reinterpret_cast<const uint32_t*>(p)[j];
  return v;
}
template <bool W16, bool ONCE>
__device__ __forceinline__ void store_piece(uint8_t* p, int n, int D, u32x4 v) {
  if (W16) {
    store_as<ONCE, u32x4>(p, v);
  } else if (n + 4 <= D) {
    store_as<ONCE, u32x4_a4>(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (n + j < D) reinterpret_cast<uint32_t*>(p)[j] = v[j];
  }
}
// Whether the streams carry the non-temporal hint.  Lines that two rows share are written in two parts, which large outputs
// then send to memory separately: 4096 rows x 17407 211 us with the hint, 164 without; 2048 rows 95 and 87; 1536 rows 71 and 73;
// 4096 rows x 17408 117 and 128.
inline bool expand_once(int M, int D) { return D % 4 == 0 || (int64_t)M * D < ((int64_t)1 << 25); }
// piece + the sums at s (4 or 8 float32), rounded to the output's type
template <bool W16>
__device__ __forceinline__ u32x4 add_piece(u32x4 v, const float* s, int ot) {
  const f32x4 a = {s[0], s[1], s[2], s[3]};
  if constexpr (!W16) {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t d = v[j];
      o[j] = __float_as_uint(__uint_as_float(d) + a[j]);
    }
    return o;
  } else {
    const f32x4 b = {s[4], s[5], s[6], s[7]};
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t d = v[j >> 1], q = (j & 1) ? d >> 16 : d & 0xFFFFu;
      const float f = (ot == X_BF16 ? bf16_bits_to_f32(q) : (float)f16_from_bits((uint16_t)q)) + (j < 4 ? a[j & 3] : b[j & 3]);
      h[j] = ot == X_BF16 ? (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f) : (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f);
    }
    return u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
  }
}

// A wave's LDS: the sums of a strip, 32 rows of float32 padded by 16 bytes (before the strips: a 32 x 32 piece of t), and the
// strip's weights of one rank step, as a transposing tile or as rows of 32 ranks.  Rows are padded by 16 bytes, which spreads the
// operand reads of 16 rows over all banks.
template <int NK> constexpr int sum_row() { return kStrip<NK> + 4; }
template <int T> constexpr int rank_row() { return 32 * esize<T>() + 16; }
template <int WT, bool TRANS, int NK> constexpr int expand_wave_lds() {
  return kRows * sum_row<NK>() * 4 + (TRANS ? terms<WT>() * tr_plane<kStrip<NK>>() : kStrip<NK> * rank_row<WT>());
}
static_assert(kRows * rank_row<X_BF16>() <= kRows * sum_row<2>() * 4, "t fits the sums' space");

// NK: rank steps of 32.  W16: out has 16-bit elements.  ONCE: the streams' hint.
template <int WT, bool TRANS, int NK, bool W16, bool ONCE>
__global__ void __launch_bounds__(256) lora_expand_kernel(int M, int D, int E, int R, int strips, int nx,
                                                          const uint16_t* __restrict__ t, const uint8_t* __restrict__ w,
                                                          const int32_t* __restrict__ ids, const uint8_t* base, uint8_t* out,
                                                          int ot) {
  constexpr int NW = terms<WT>();
  constexpr int ES = W16 ? 2 : 4, PE = 16 / ES;          // elements of a 16-byte piece
  constexpr int SW = kStrip<NK>, Q = SW / 16;            // MFMA column blocks of a strip
  constexpr int PL = SW / PE, PN = kRows * PL / 64;      // pieces of a row, pieces per lane
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int rt = (int)blockIdx.x / nx;
  const int m0 = rt * kRows;
  const int n_begin = (((int)blockIdx.x - rt * nx) * 4 + wave) * SW * strips, n_end = min(n_begin + SW * strips, D);
  const int id = tile_id(ids, m0, M, E);
  uint32_t lead = tile_leaders(id);
  float* sums = reinterpret_cast<float*>(lds + wave * expand_wave_lds<WT, TRANS, NK>());
  uint8_t* tile = reinterpret_cast<uint8_t*>(sums + kRows * sum_row<NK>());

  // the strip's pieces of the rows whose bit in `rows` is set: piece q covers row c / PL, elements PE (c % PL) .., c = lane + 64 q
  u32x4 y[PN];
  auto load_rows = [&](uint32_t rows, int n0) {
#pragma unroll
    for (int q = 0; q < PN; ++q) {
      const int c = lane + 64 * q, row = c / PL, n = n0 + PE * (c % PL);
      y[q] = u32x4{0u, 0u, 0u, 0u};
      if (base != nullptr && (rows >> row & 1) && n < n_end)
        y[q] = load_piece<W16, ONCE>(base + ((size_t)(m0 + row) * D + n) * ES, n, D);
    }
  };
  auto store_rows = [&](uint32_t rows, int n0, const u32x4* v) {
#pragma unroll
    for (int q = 0; q < PN; ++q) {
      const int c = lane + 64 * q, row = c / PL, n = n0 + PE * (c % PL);
      if ((rows >> row & 1) && n < n_end) store_piece<W16, ONCE>(out + ((size_t)(m0 + row) * D + n) * ES, n, D, v[q]);
    }
  };
  // rows without an adapter: out = base
  const uint32_t bare = (uint32_t)__ballot(id < 0 && m0 + (lane & 31) < M);
  if (blockIdx.z == 0 && bare != 0 && base != out) {
    for (int n0 = n_begin; n0 < n_end; n0 += SW) {
      load_rows(bare, n0);
      store_rows(bare, n0, y);
    }
  }

  for (int z = 0; lead != 0; ++z, lead &= lead - 1) {
    if (z % (int)gridDim.z != (int)blockIdx.z) continue;
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctz(lead));
    const uint32_t mask = tile_mask(id, e);
    const uint8_t* we = w + (size_t)e * R * D * esize<WT>();
    // a rank step's weights of a strip in whole lines.  TRANS: rows r of D elements, chunks of 8 of the 32 x strip tile; else
    // rows n of R, 16-byte pieces of the 32 ranks
    constexpr int WP = 16 / esize<WT>(), WL = 32 / WP, WN = TRANS ? 1 : SW * WL / 64;
    Raw<WT> raw[Q];
    u32x4 wr[WN];
    auto load_w = [&](int n0, int k) {
      if constexpr (TRANS) {
        constexpr int CW = SW / 8;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int c = lane + 64 * q, r = 32 * k + c / CW, n = n0 + 8 * (c % CW);
          if (r < R && n < D) raw_load<WT, true>(we + ((size_t)r * D + n) * esize<WT>(), raw[q]);
          else raw_zero(raw[q]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < WN; ++q) {
          const int c = lane + 64 * q, n = n0 + c / WL, r = 32 * k + WP * (c % WL);
          wr[q] = r < R && n < D ? *reinterpret_cast<const u32x4*>(we + ((size_t)n * R + r) * esize<WT>()) : u32x4{0u, 0u, 0u, 0u};
        }
      }
    };
    if (n_begin < n_end) {
      load_w(n_begin, 0);
      load_rows(mask, n_begin);
    }
    // t of the two 16-row blocks: lane holds row l16 of the block, ranks 32 k + 8 g .. + 7; loaded in whole lines, 2 pieces of
    // 8 ranks per lane, and turned in LDS
    bf16x8 tf[2][NK][3];
    uint8_t* tt = reinterpret_cast<uint8_t*>(sums);
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      u32x4 tr[3][2];
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = lane + 64 * h, row = c >> 2, r = 32 * k + 8 * (c & 3);
          tr[q][h] = (mask >> row & 1) && r < R
                         ? *reinterpret_cast<const u32x4*>(t + (size_t)q * M * R + (size_t)(m0 + row) * R + r)
                         : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        wave_lds_fence();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = lane + 64 * h;
          *reinterpret_cast<u32x4*>(tt + (c >> 2) * rank_row<X_BF16>() + (c & 3) * 16) = tr[q][h];
        }
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          tf[i][k][q] = *reinterpret_cast<const bf16x8*>(tt + (16 * i + l16) * rank_row<X_BF16>() + 16 * g);
      }
    }

    for (int n0 = n_begin; n0 < n_end; n0 += SW) {
      f32x4 acc[Q][2];
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[q][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        wave_lds_fence();
        if constexpr (TRANS) {
#pragma unroll
          for (int q = 0; q < Q; ++q) tr_write<WT, SW>(tile, lane + 64 * q, raw[q]);
        } else {
#pragma unroll
          for (int q = 0; q < WN; ++q) {
            const int c = lane + 64 * q;
            *reinterpret_cast<u32x4*>(tile + (c / WL) * rank_row<WT>() + (c % WL) * 16) = wr[q];
          }
        }
        wave_lds_fence();
        // the next weights (this strip's next rank step, or the next strip's first) fly during the MFMAs
        if (k + 1 < NK) load_w(n0, k + 1);
        else if (n0 + SW < n_end) load_w(n0 + SW, 0);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          bf16x8 wf[NW];
          if constexpr (TRANS) {
            tr_read<SW, NW>(tile, q, wf);
          } else {
            Raw<WT> r;
            const uint8_t* p = tile + (16 * q + l16) * rank_row<WT>() + 8 * g * esize<WT>();
            r.v[0] = *reinterpret_cast<const u32x4*>(p);
            if constexpr (WT == X_F32) r.v[1] = *reinterpret_cast<const u32x4*>(p + 16);
            raw_terms<WT>(r, wf);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[q][i] = mfma_terms<NW, 3>(wf, tf[i][k], acc[q][i]);
        }
      }
      // the sums, MFMA rows = n: lane holds columns 16 q + 4 g .. + 3 of row 16 i + l16
      wave_lds_fence();
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<f32x4*>(sums + (16 * i + l16) * sum_row<NK>() + 16 * q + 4 * g) = acc[q][i];
      wave_lds_fence();
      u32x4 o[PN];
#pragma unroll
      for (int q = 0; q < PN; ++q) {
        const int c = lane + 64 * q;
        o[q] = add_piece<W16>(y[q], sums + (c / PL) * sum_row<NK>() + PE * (c % PL), ot);
      }
      if (n0 + SW < n_end) load_rows(mask, n0 + SW);
      store_rows(mask, n0, o);
    }
  }
}

// Few rows, forward: a workgroup takes one row and kRowCols columns.  The ranks of one n lie next to each other in b; G
// lanes (a power of two covering R / 8) share an n, each holding its 8 ranks of t in registers, so a wave reads b in whole
// lines; their float32 sums meet in log2 G exchanges.
constexpr int kRowCols = 256;

template <int WT, int G>
__global__ void __launch_bounds__(256) lora_expand_rows_kernel(int M, int N, int E, int R, int nx, const uint16_t* __restrict__ t,
                                                               const uint8_t* __restrict__ w, const int32_t* __restrict__ ids,
                                                               const float* base, float* out) {
  constexpr int NPW = 64 / G;                    // columns of a wave's step
  constexpr int STEPS = kRowCols / (4 * NPW);    // steps of a wave
  constexpr int U = STEPS < 8 ? STEPS : 8;       // of which are in flight
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = (int)blockIdx.x / nx, n0 = ((int)blockIdx.x - m * nx) * kRowCols + wave * (kRowCols / 4);
  const int e = ids[m];
  const float* yr = base ? base + (size_t)m * N : nullptr;
  float* o = out + (size_t)m * N;
  if (e < 0 || e >= E) {
    if (base != out) {
      const int n = n0 + lane;
      if (n < N) o[n] = yr ? yr[n] : 0.f;
    }
    return;
  }
  const int c = lane % G, ln = lane / G;
  const bool on = 8 * c < R;
  float tr[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const uint8_t* we = w + ((size_t)e * N * R + 8 * c) * esize<WT>();
  const uint16_t* p = t + (size_t)m * R + 8 * c;
  u32x4 th[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) th[q] = on ? *reinterpret_cast<const u32x4*>(p + q * (size_t)M * R) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int s = 0; s < STEPS; s += U) {
    Raw<WT> raw[U];
    float y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + (s + u) * NPW + ln;
      raw_zero(raw[u]);
      if (on && n < N) raw_load<WT, true>(we + (size_t)n * R * esize<WT>(), raw[u]);
      y[u] = yr && c == 0 && n < N ? yr[n] : 0.f;
    }
    if (s == 0) {
#pragma unroll
      for (int q = 2; q >= 0; --q) {             // the terms of t, smallest first: exact sums
        float v[8];
        Raw<X_BF16> r{{th[q]}};
        raw_f32<X_BF16>(r, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) tr[j] += v[j];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + (s + u) * NPW + ln;
      float v[8], a = 0.f;
      raw_f32<WT>(raw[u], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) a = fmaf(tr[j], v[j], a);
#pragma unroll
      for (int off = G / 2; off >= 1; off >>= 1) a += __shfl_xor(a, off, 64);
      if (c == 0 && n < N) o[n] = y[u] + a;
    }
  }
}

// Few rows of a small adapter, forward in one launch: every workgroup computes its row's t for itself (a wave per rank, as
// lora_shrink_rows_kernel does), which costs less than a second launch while the adapter's K x R matrix is small.
template <int XT, int WT>
__global__ void __launch_bounds__(256) lora_rows_kernel(int M, int K, int N, int E, int R, int nx, const uint8_t* __restrict__ x,
                                                        const uint8_t* __restrict__ a, const uint8_t* __restrict__ b,
                                                        const float* __restrict__ scale, const int32_t* __restrict__ ids,
                                                        const float* base, float* out) {
  __shared__ float t[WQ_LORA_MAX_RANK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = (int)blockIdx.x / nx, n = ((int)blockIdx.x - m * nx) * 256 + (int)threadIdx.x;
  const int e = ids[m];
  float y = 0.f;
  if (base != nullptr && n < N) y = base[(size_t)m * N + n];
  if (e >= 0 && e < E) {
    const uint8_t* xr = x + (size_t)m * K * esize<XT>();
    const float f = scale[e];
    for (int r = wave; r < R; r += 8) {        // two ranks at a time (R is a multiple of 8)
      const uint8_t* a0 = a + ((size_t)e * R + r) * K * esize<WT>();
      const uint8_t* a1 = a0 + (size_t)4 * K * esize<WT>();
      float s0 = 0.f, s1 = 0.f;
      for (int k = 8 * lane; k < K; k += 512) {
        Raw<XT> rx;
        Raw<WT> r0, r1;
        raw_load<XT, true>(xr + (size_t)k * esize<XT>(), rx);
        raw_load<WT, true>(a0 + (size_t)k * esize<WT>(), r0);
        raw_load<WT, true>(a1 + (size_t)k * esize<WT>(), r1);
        float u[8], v[8], w[8];
        raw_f32<XT>(rx, u);
        raw_f32<WT>(r0, v);
        raw_f32<WT>(r1, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s0 = fmaf(u[j], v[j], s0);
          s1 = fmaf(u[j], w[j], s1);
        }
      }
      s0 = wave64_sum(s0);
      s1 = wave64_sum(s1);
      if (lane == 0) {
        t[r] = s0 * f;
        t[r + 4] = s1 * f;
      }
    }
    __syncthreads();
    if (n < N) {
      const uint8_t* br = b + ((size_t)e * N + n) * R * esize<WT>();
      float acc = 0.f;
      for (int r = 0; r < R; r += 8) {
        Raw<WT> raw;
        raw_load<WT, true>(br + (size_t)r * esize<WT>(), raw);
        float v[8];
        raw_f32<WT>(raw, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc = fmaf(t[r + j], v[j], acc);
      }
      y += acc;
    }
  }
  if (n < N) out[(size_t)m * N + n] = y;
}

// Few rows, backward: a workgroup takes one row and 2048 columns, a thread 8 of them: all ranks' pieces of a, read in whole
// lines, times t from LDS.
template <int WT>
__global__ void __launch_bounds__(256) lora_expand_rows_t_kernel(int M, int D, int E, int R, int nx, const uint16_t* __restrict__ t,
                                                                 const uint8_t* __restrict__ w, const int32_t* __restrict__ ids,
                                                                 const uint8_t* base, uint8_t* out, int ot) {
  __shared__ float tr[256];
  const int m = (int)blockIdx.x / nx, n = (((int)blockIdx.x - m * nx) * 256 + (int)threadIdx.x) * 8;
  const int e = ids[m];
  const int es = ot == X_F32 ? 4 : 2;
  const size_t at = ((size_t)m * D + n) * es;
  u32x4 y[2] = {u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
  if (base != nullptr && n < D) {              // D is a multiple of 16
    y[0] = *reinterpret_cast<const u32x4*>(base + at);
    if (ot == X_F32) y[1] = *reinterpret_cast<const u32x4*>(base + at + 16);
  }
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (e >= 0 && e < E) {
    if ((int)threadIdx.x < R) {
      const uint16_t* p = t + (size_t)m * R + threadIdx.x;
      tr[threadIdx.x] = (bf16_bits_to_f32(p[2 * (size_t)M * R]) + bf16_bits_to_f32(p[(size_t)M * R])) + bf16_bits_to_f32(p[0]);
    }
    __syncthreads();
    if (n < D) {
      const uint8_t* we = w + ((size_t)e * R * D + n) * esize<WT>();
      for (int r = 0; r < R; r += 8) {         // R is a multiple of 8
        Raw<WT> raw[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) raw_load<WT, true>(we + (size_t)(r + q) * D * esize<WT>(), raw[q]);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float v[8];
          raw_f32<WT>(raw[q], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = fmaf(tr[r + q], v[j], acc[j]);
        }
      }
    }
  }
  if (n >= D) return;
  if (ot == X_F32) {
    *reinterpret_cast<u32x4*>(out + at) = add_piece<false>(y[0], acc, ot);
    *reinterpret_cast<u32x4*>(out + at + 16) = add_piece<false>(y[1], acc + 4, ot);
  } else {
    *reinterpret_cast<u32x4*>(out + at) = add_piece<true>(y[0], acc, ot);
  }
}

template <int WT, bool TRANS, int NK, bool W16, bool ONCE = true>
hipError_t go(int M, int D, int E, int R, const uint16_t* t, const void* w, const int32_t* ids, const void* base, void* out,
              int ot, hipStream_t st) {
  if constexpr (!TRANS && ONCE) {                        // transposed: D is a multiple of 16
    if (!expand_once(M, D)) return go<WT, TRANS, NK, W16, false>(M, D, E, R, t, w, ids, base, out, ot, st);
  }
  constexpr int lds = 4 * expand_wave_lds<WT, TRANS, NK>();
  if (!raise_lds_limit<lora_expand_kernel<WT, TRANS, NK, W16, ONCE>>()) return hipErrorInvalidValue;
  const int tiles = (M + kRows - 1) / kRows;
  // strips per wave: more while the launch keeps over 2048 workgroups (t is loaded once per wave)
  constexpr int kGroup = 4 * kStrip<NK>;
  int strips = 1;
  while (strips < 256 / kStrip<NK> && (int64_t)tiles * ((D + 2 * strips * kGroup - 1) / (2 * strips * kGroup)) > 2048) strips *= 2;
  const int nx = (D + strips * kGroup - 1) / (strips * kGroup);
  const int dz = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(E, kRows), 2048 / ((int64_t)tiles * nx)));
  hipLaunchKernelGGL((lora_expand_kernel<WT, TRANS, NK, W16, ONCE>), dim3((unsigned)(tiles * nx), 1, dz), dim3(256), lds, st, M, D, E, R,
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

template <int WT, int G>
hipError_t go_rows(int M, int N, int E, int R, const uint16_t* t, const void* w, const int32_t* ids, const void* base, void* out,
                   hipStream_t st) {
  const int nx = (N + kRowCols - 1) / kRowCols;
  hipLaunchKernelGGL((lora_expand_rows_kernel<WT, G>), dim3((unsigned)(M * nx)), dim3(256), 0, st, M, N, E, R, nx, t,
                     reinterpret_cast<const uint8_t*>(w), ids, reinterpret_cast<const float*>(base), reinterpret_cast<float*>(out));
  return hipGetLastError();
}
template <int WT, typename... A>
hipError_t rows_by_rank(int M, int N, int E, int R, A... a) {
  if (R <= 8) return go_rows<WT, 1>(M, N, E, R, a...);
  if (R <= 16) return go_rows<WT, 2>(M, N, E, R, a...);
  if (R <= 32) return go_rows<WT, 4>(M, N, E, R, a...);
  if (R <= 64) return go_rows<WT, 8>(M, N, E, R, a...);
  if (R <= 128) return go_rows<WT, 16>(M, N, E, R, a...);
  return go_rows<WT, 32>(M, N, E, R, a...);
}

}  // namespace

// One launch while an adapter's a has at most 8192 elements and all workgroups together read at most 4 Mi of them.
bool lora_one_launch(int M, int K, int N, int R) {
  const int64_t each = (int64_t)K * R;
  return each <= 8192 && each * M * ((N + 255) / 256) <= (4 << 20);
}
hipError_t lora_rows(int M, int K, int N, int E, int R, const void* x, XType xt, const void* a, const void* b, XType wt,
                     const float* scale, const int32_t* ids, const float* y, float* out, hipStream_t st) {
  const int nx = (N + 255) / 256;
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(M * nx)), dim3(256), 0, st, M, K, N, E, R, nx, reinterpret_cast<const uint8_t*>(x),
                       reinterpret_cast<const uint8_t*>(a), reinterpret_cast<const uint8_t*>(b), scale, ids, y, out);
    return hipGetLastError();
  };
  switch (3 * (int)xt + (int)wt) {
    case 0: return launch(lora_rows_kernel<X_F32, X_F32>);
    case 1: return launch(lora_rows_kernel<X_F32, X_BF16>);
    case 2: return launch(lora_rows_kernel<X_F32, X_F16>);
    case 3: return launch(lora_rows_kernel<X_BF16, X_F32>);
    case 4: return launch(lora_rows_kernel<X_BF16, X_BF16>);
    case 5: return launch(lora_rows_kernel<X_BF16, X_F16>);
    case 6: return launch(lora_rows_kernel<X_F16, X_F32>);
    case 7: return launch(lora_rows_kernel<X_F16, X_BF16>);
    default: return launch(lora_rows_kernel<X_F16, X_F16>);
  }
}

// Forward (not trans) the output is float32, backward any type.
hipError_t lora_expand(bool few, int M, int D, int E, int R, const uint16_t* t, const void* w, XType wt, bool trans,
                       const int32_t* ids, const void* base, void* out, XType ot, hipStream_t st) {
  if (trans && few) {
    const int nx = (D + 2047) / 2048;
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(M * nx)), dim3(256), 0, st, M, D, E, R, nx, t, reinterpret_cast<const uint8_t*>(w),
                         ids, reinterpret_cast<const uint8_t*>(base), reinterpret_cast<uint8_t*>(out), (int)ot);
      return hipGetLastError();
    };
    if (wt == X_F32) return launch(lora_expand_rows_t_kernel<X_F32>);
    if (wt == X_BF16) return launch(lora_expand_rows_t_kernel<X_BF16>);
    return launch(lora_expand_rows_t_kernel<X_F16>);
  }
  if (!trans && ot == X_F32 && few) {
    if (wt == X_F32) return rows_by_rank<X_F32>(M, D, E, R, t, w, ids, base, out, st);
    if (wt == X_BF16) return rows_by_rank<X_BF16>(M, D, E, R, t, w, ids, base, out, st);
    return rows_by_rank<X_F16>(M, D, E, R, t, w, ids, base, out, st);
  }
  if (!trans) return ot == X_F32 ? by_weight<false, false>(wt, M, D, E, R, t, w, ids, base, out, (int)ot, st) : hipErrorInvalidValue;
  if (ot == X_F32) return by_weight<true, false>(wt, M, D, E, R, t, w, ids, base, out, (int)ot, st);
  return by_weight<true, true>(wt, M, D, E, R, t, w, ids, base, out, (int)ot, st);
}

}  // namespace wq
