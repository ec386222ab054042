// Device-side pieces shared by the low-rank adapter kernels (lora_*.hip).
//
// Operand terms.  The adapters' products run on bfloat16 MFMAs but are to be float32 products: every operand is
// taken as a sum of bfloat16 terms that holds all its bits (down to 2^-133, bfloat16's smallest step) -- bfloat16 is 1 term,
// float16 2, float32 (and the float32 intermediates) 3 -- and a product is the sum of the term products that reach above 2^-25 of it (term indices i + j
// <= 2).  The kernels move far more bytes than they multiply, so the extra MFMAs hide behind the loads.
//
// Transposed operands.  An MFMA 16x16x32 operand wants 8 consecutive contraction indices per lane.  Where memory
// holds the other index contiguous, a wave writes its 32 x C tile of terms to LDS as it came and reads it with
// ds_read_b64_tr_b16: within 16 lanes, lane i receives column i of 4 rows of 16 elements.
#pragma once
#include "dev_common.h"
#include "launch.h"

namespace wq {
namespace lora {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kRows = 32;            // rows of the row tiles (two 16-row MFMA blocks)

template <int T> constexpr int terms() { return T == X_F32 ? 3 : (T == X_F16 ? 2 : 1); }
template <int T> constexpr int esize() { return T == X_F32 ? 4 : 2; }

// 8 elements as loaded.
template <int T> struct Raw { u32x4 v[T == X_F32 ? 2 : 1]; };

template <int T>
__device__ __forceinline__ void raw_zero(Raw<T>& r) {
  r.v[0] = u32x4{0u, 0u, 0u, 0u};
  if constexpr (T == X_F32) r.v[1] = u32x4{0u, 0u, 0u, 0u};
}
// ALIGNED: p is 16-byte aligned; else it is aligned to an element.
template <int T, bool ALIGNED>
__device__ __forceinline__ void raw_load(const uint8_t* p, Raw<T>& r) {
  if constexpr (ALIGNED) {
    r.v[0] = *reinterpret_cast<const u32x4*>(p);
    if constexpr (T == X_F32) r.v[1] = *reinterpret_cast<const u32x4*>(p + 16);
  } else if constexpr (T == X_F32) {
    r.v[0] = *reinterpret_cast<const u32x4_a4*>(p);
    r.v[1] = *reinterpret_cast<const u32x4_a4*>(p + 16);
  } else {
    r.v[0] = *reinterpret_cast<const u32x4_a2*>(p);
  }
}
// The first n (< 8) elements at p, zeros behind them.
template <int T>
__device__ __forceinline__ void raw_load_part(const uint8_t* p, int n, Raw<T>& r) {
  raw_zero(r);
  if constexpr (T == X_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) r.v[j >> 2][j & 3] = reinterpret_cast<const uint32_t*>(p)[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) r.v[0][j >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j & 1));
  }
}

// N float32 values -> 3 bfloat16 terms each (round to nearest, exact remainders).
template <int N, typename V>
__device__ __forceinline__ void split3(const float* v, V* t) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const __bf16 hi = (__bf16)v[j];
    const float r1 = v[j] - (float)hi;
    const __bf16 mid = (__bf16)r1;
    t[0][j] = hi;
    t[1][j] = mid;
    t[2][j] = (__bf16)(r1 - (float)mid);
  }
}

template <int T>
__device__ __forceinline__ void raw_terms(const Raw<T>& r, bf16x8* t) {
  if constexpr (T == X_BF16) {
    t[0] = __builtin_bit_cast(bf16x8, r.v[0]);
  } else if constexpr (T == X_F16) {
    const f16x8 h = __builtin_bit_cast(f16x8, r.v[0]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = (float)h[j];
      const __bf16 hi = (__bf16)v;
      t[0][j] = hi;
      t[1][j] = (__bf16)(v - (float)hi);
    }
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r.v[j >> 2][j & 3]);
    split3<8>(v, t);
  }
}

template <int T>
__device__ __forceinline__ void raw_f32(const Raw<T>& r, float* v) {
  if constexpr (T == X_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r.v[j >> 2][j & 3]);
  } else if constexpr (T == X_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t d = r.v[0][j];
      v[2 * j] = __uint_as_float(d << 16);
      v[2 * j + 1] = __uint_as_float(d & 0xFFFF0000u);
    }
  } else {
    const f16x8 h = __builtin_bit_cast(f16x8, r.v[0]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)h[j];
  }
}

// acc += sum of the term products a[i] b[j], i + j <= 2.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma_terms(const bf16x8* a, const bf16x8* b, f32x4 acc) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)          // small products first
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j <= 2) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc, 0, 0, 0);
  return acc;
}

// ---- a wave's transposing LDS tile: 32 contraction rows x C columns, one plane per term ---------------------------
// Row strides that put the 16 rows x 32 bytes of a read on all banks twice (the least it takes).
template <int C> constexpr int tr_stride() { return C == 16 ? 32 : 2 * C + 32; }
template <int C> constexpr int tr_plane() { return 32 * tr_stride<C>(); }

// Columns 16 c .. 16 c + 15 as an operand: lane holds column lane % 16, rows 8 (lane / 16) .. + 7.
template <int C, int NT>
__device__ __forceinline__ void tr_read(const uint8_t* tile, int c, bf16x8* t) {
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const uint8_t* p = tile + (8 * g + (l >> 2)) * tr_stride<C>() + 32 * c + 8 * (l & 3);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + i * tr_plane<C>()));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + i * tr_plane<C>() + 4 * tr_stride<C>()));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    t[i] = __builtin_bit_cast(bf16x8, s16x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
  }
}

// Chunk q (of 32 C / 8) of a tile of typed elements: row q / (C / 8), columns 8 (q % (C / 8)) .. + 7.
template <int T, int C>
__device__ __forceinline__ void tr_write(uint8_t* tile, int q, const Raw<T>& r) {
  bf16x8 t[terms<T>()];
  raw_terms<T>(r, t);
  uint8_t* p = tile + (q / (C / 8)) * tr_stride<C>() + (q % (C / 8)) * 16;
#pragma unroll
  for (int i = 0; i < terms<T>(); ++i) *reinterpret_cast<bf16x8*>(p + i * tr_plane<C>()) = t[i];
}

// ---- rows and their adapters ---------------------------------------------------------------------------------------
// Adapter of row m0 + lane % 32, -1 where there is none.
__device__ __forceinline__ int tile_id(const int32_t* ids, int m0, int M, int E) {
  const int m = m0 + (threadIdx.x & 31);
  const int e = m < M ? ids[m] : -1;
  return e >= 0 && e < E ? e : -1;
}
// Bit i: row i is the first of the 32 that names its adapter.  Scalar masks throughout: written as a condition per lane, the
// 31 comparisons became 31 nested branches.
__device__ __forceinline__ uint32_t tile_leaders(int id) {
  if (__ballot(id != __builtin_amdgcn_readfirstlane(id)) == 0) return id >= 0 ? 1u : 0u;   // one adapter, or none
  uint32_t later = 0;                        // rows whose adapter an earlier row names
#pragma unroll
  for (int j = 0; j < 31; ++j) later |= (uint32_t)__ballot(id == __builtin_amdgcn_readlane(id, j)) & (~1u << j);
  return (uint32_t)__ballot(id >= 0) & ~later;
}
// Rows of the tile with adapter e.
__device__ __forceinline__ uint32_t tile_mask(int id, int e) { return (uint32_t)__ballot(id == e); }

}  // namespace lora

// Whether a batch takes the row kernels (one row at a time, every row reading its adapter) instead of the tiles: while what
// all rows read of their adapters, from L2, stays below 300 MB and the work small.  At 5120 -> 17408 in bfloat16, all rows on one
// adapter (the tiles' best case), rank 16: 128 rows 14 us against 19, 256 rows 24 against 21, 512 rows 42 against 30; rank 64: 64
// rows 16 against 21, 128 rows 27 against 24; each row on a random adapter, rank 16: 256 rows 26 against 101, 512 rows 43
// against 172.
inline bool lora_few_rows(int M, int K, int N, int R, XType wt) {
  const int64_t mr = (int64_t)M * (R < 16 ? 16 : R);
  return mr <= 16384 && mr * ((int64_t)K + N) * (wt == X_F32 ? 4 : 2) <= 300000000;
}

// Launchers of the three products (internal to the lora files).  The rank-R intermediate is held as its operand
// terms, t [3][M][R] bfloat16 of scale[e] * sum, so that the many workgroups that read it neither add nor split it;
// rows without an adapter are not written.
// t = scale[e] * sum_d x[m,d] w[e][r,d] (trans: w[e][d,r]), e = ids[m]; few: by rows (lora_few_rows); parts: scratch of
// lora_shrink_bytes.
hipError_t lora_shrink(bool few, int M, int D, int E, int R, const void* x, XType xt, const void* w, XType wt, bool trans,
                       const float* scale, const int32_t* ids, uint16_t* t, float* parts, hipStream_t st);
size_t lora_shrink_bytes(int M, int D, int R, XType xt);
// out[m,n] = base[m,n] + sum_r t[m,r] w[e][n,r] (trans: w[e][r,n]); base may be null or out.
hipError_t lora_expand(bool few, int M, int D, int E, int R, const uint16_t* t, const void* w, XType wt, bool trans,
                       const int32_t* ids, const void* base, void* out, XType ot, hipStream_t st);
// Both forward products in one launch, for small adapters.
bool lora_one_launch(int M, int K, int N, int R);
hipError_t lora_rows(int M, int K, int N, int E, int R, const void* x, XType xt, const void* a, const void* b, XType wt,
                     const float* scale, const int32_t* ids, const float* y, float* out, hipStream_t st);
// g[e][r,d] (rcontig: g[e][d,r]) = sum_{m: ids[m] = e} t[m,r] v[m,d], one or two such sums over v of one type; parts: scratch
// of lora_outer_bytes, which lora_outer_join (with any one or two jobs run before) adds up.
struct OuterJob {
  int D;
  const uint16_t* t;
  const void* v;
  XType vt;
  bool rcontig;
  float* g;
  float* parts;
};
hipError_t lora_outer(int M, int E, int R, const OuterJob* jobs, int count, const int32_t* ids, hipStream_t st);
hipError_t lora_outer_join(int M, int E, int R, const OuterJob* jobs, int count, hipStream_t st);
size_t lora_outer_bytes(int M, int D, int E, int R);

}  // namespace wq
