// Gradient of a quantised linear with respect to its input (gfx950): qlinear_backward in
// include/wqmlp_adapters.h and awq_linear_backward in include/wqmlp_blocks.h,  dx[m,k] = sum_n dy[m,n] dq(W[n,k]).
//
// A GEMM whose contraction runs over the weight's rows, while the weights are packed along their columns (k), so
// the matrix cores need each lane to hold 8 consecutive n of one column: the transpose of what is stored.  The
// packed bytes are transposed on their way out of LDS (ds_read_b64_tr_b8: within 16 lanes, lane i receives byte
// column i of 8 rows of 16 bytes), before they are decoded, so the transpose moves 1 byte per FP8 weight and half
// a byte per NVFP4 weight, and every weight is decoded once per tile row, in registers.
//   FP8: one read gives a fragment's 8 codes; the channel scale s[n] runs along the contraction, so it is
//     multiplied into dy beforehand.
//   NVFP4: a byte column holds the k pair (2c, 2c+1), so one read gives both column blocks of a wave, the even
//     and the odd k.  The E4M3 group scales (one per n and 16 k) are held in LDS as float16, [group][n], so a
//     lane's 8 scales are one 16-byte read; E2M1 x E4M3 products are exact float16 values.
//   AWQ: byte columns as NVFP4; scales and biases (one each per n and 32 k) are held the same way.  A transposed dword
//     holds the nibbles of n .. n + 3, which masks leave alone in their bytes as E4M3 codes of 0 .. 15.
//
// Tile: 4 waves compute (32 MB / TERMS) rows x 256 columns, 64 columns per wave; the waves share the activation
// tile (64 n of float16 = 128-byte rows, moved by global->LDS copies), each decodes only its own columns.  n is
// walked in steps of 64 through a two-stage ring; the one barrier of a step sits after the last LDS read of its
// stage, the copies for two steps ahead follow it, and the first fragments of the next step are read behind the
// last MFMAs of this one.  Two workgroups share a CU.
//
// The matrix cores bound it.  Calls in a row, bfloat16 dx: NVFP4 4096 x 5120 -> 17408 690-720 us (1.01-1.06 PFLOP/s; a float16
// product of those sizes in the library 635), FP8 512 x 17408 -> 5120 107-110 us, of which the GEMM 85-87 (1.05-1.07 PFLOP/s) and
// the kernels before and after it 20.  float32 dx, twice the MFMAs: NVFP4 2048 x 5120 -> 17408 685 us (1.07 PFLOP/s in MFMAs), FP8
// 512 x 17408 -> 5120 193 us.  In the first two MFMAs are busy in
// 55% and 59% of the busy CUs' cycles; 5.9 and 3.3 VALU instructions per MFMA (the decode) and the weights' LDS reads take turns
// with them.  AWQ 1024 x 17408 -> 5120 227-230 us (0.80 PFLOP/s; the library's product 225), of which dy's preparation 14, the GEMM
// 205 in 3 parts of 160 tiles, MFMAs busy in 48% of its cycles, and the parts' sum 12; 129 x 67 -> 320 float32 13 us a call.
//
// Numerics: dy (times s[n] for FP8, one float32 rounding) is scaled per row by a power of two so that its largest
// finite magnitude lies in [2^14, 2^15).  TERMS = 1 (bfloat16 dx): rounded once to float16, off by at most 2^-11 of the
// element, where dx's own rounding is 2^-8, or by half of float16's smallest step, 2^-39 of the row's largest.  TERMS = 2
// (float32 dx): the float16 value and, as another float16, 2^12 times what it left, so that the second term of a small
// element beside a large one is not lost among the subnormals: off by at most 2^-22 of the element or 2^-51 of the row's
// largest.  The second terms' products have float32 accumulators of their own (a tile of two terms has half the rows, so
// both kinds of tile hold as many), which join the others' at the end.
#include <algorithm>
#include <type_traits>

#include "dev_common.h"
#include "launch.h"

namespace wq {

namespace {

// ---- dy -> float16 terms ---------------------------------------------------------------------------------------
// What float16 h left of x, times 2^12; nothing where h is infinite (x - h would be NaN, and the row's infinities lose their
// sign) or NaN.  |x| < 2^15, so h is off by at most 8.
constexpr float kSecond = 4096.f;
__device__ __forceinline__ _Float16 second_term(float x, _Float16 h) {
  const float r = (x - (float)h) * kSecond;
  return r == r ? (_Float16)r : (_Float16)0.f;
}

// One workgroup per row of dy [M][N] (any N, so rows are only element-aligned): the row's largest finite magnitude, then the scaled
// float16 terms, [TERMS][M][Np] with zeros from N to Np (a multiple of 64).  A thread keeps RC chunks of 8 elements in registers,
// loaded without a branch between them so that all are in flight at once; longer rows read the rest twice.  The up to 7 elements
// behind the last whole chunk are one thread's.
template <bool BF, bool SC, int TERMS, int RC>
__global__ void __launch_bounds__(256) grad_prep_kernel(int M, int N, int Np, const void* __restrict__ dy,
                                                        const float* __restrict__ scale, uint16_t* __restrict__ a16,
                                                        float* __restrict__ rowscale) {
  typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
  typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
  __shared__ float wmax[4];
  const int m = (int)blockIdx.x, t = (int)threadIdx.x;
  const uint8_t* row = reinterpret_cast<const uint8_t*>(dy) + (size_t)m * N * (BF ? 2 : 4);
  const int nf = N / 8;                          // whole chunks
  struct Chunk { u32x4 v[BF ? 1 : 2]; f32x4 s[SC ? 2 : 1]; };
  auto load = [&](int c, Chunk& d) {             // c < nf
    if constexpr (BF) {
      d.v[0] = *reinterpret_cast<const u32x4_a2*>(row + 16 * (size_t)c);
    } else {
      d.v[0] = *reinterpret_cast<const u32x4_a4*>(row + 32 * (size_t)c);
      d.v[1] = *reinterpret_cast<const u32x4_a4*>(row + 32 * (size_t)c + 16);
    }
    if constexpr (SC) {
      d.s[0] = reinterpret_cast<const f32x4*>(scale)[2 * c];
      d.s[1] = reinterpret_cast<const f32x4*>(scale)[2 * c + 1];
    }
  };
  auto values = [&](const Chunk& d, float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = d.v[0][j];
      if constexpr (BF) {
        v[2 * j] = __uint_as_float(u << 16);
        v[2 * j + 1] = __uint_as_float(u & 0xFFFF0000u);
      } else {
        const uint32_t w = d.v[1][j];
        v[j] = __uint_as_float(u);
        v[4 + j] = __uint_as_float(w);
      }
    }
    if constexpr (SC) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= d.s[j >> 2][j & 3];
    }
  };
  uint16_t* o = a16 + (size_t)m * Np;
  auto put = [&](int c, const float* v, int e) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x0 = ldexpf(v[2 * j], -e), x1 = ldexpf(v[2 * j + 1], -e);
      const _Float16 h0 = (_Float16)x0, h1 = (_Float16)x1;
      hi[j] = as_u32(f16x2{h0, h1});
      if constexpr (TERMS == 2) lo[j] = as_u32(f16x2{second_term(x0, h0), second_term(x1, h1)});
    }
    reinterpret_cast<u32x4*>(o)[c] = u32x4{hi[0], hi[1], hi[2], hi[3]};
    if constexpr (TERMS == 2) reinterpret_cast<u32x4*>(o + (size_t)M * Np)[c] = u32x4{lo[0], lo[1], lo[2], lo[3]};
  };
  float amax = 0.f, keep[RC][8], rest = 0.f;
  auto maximum = [&](const float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(v[j]));
  };
  if (t < N - 8 * nf) {                          // element 8 nf + t
    const int n = 8 * nf + t;
    rest = BF ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(row)[n]) : reinterpret_cast<const float*>(row)[n];
    if constexpr (SC) rest *= scale[n];
    amax = finite_abs(rest);
  }
  if (nf > 0) {
    Chunk raw[RC];
#pragma unroll
    for (int i = 0; i < RC; ++i) load(min(t + 256 * i, nf - 1), raw[i]);   // past the end: the last one again, not used
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      values(raw[i], keep[i]);
      maximum(keep[i]);
    }
    for (int c = t + 256 * RC; c < nf; c += 256) {
      float v[8];
      load(c, raw[0]);
      values(raw[0], v);
      maximum(v);
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
  if ((t & 63) == 0) wmax[t >> 6] = amax;
  __syncthreads();
  const int e = f16_row_exp(fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])));
  if (t == 0) rowscale[m] = ldexpf(1.0f, e);
#pragma unroll
  for (int i = 0; i < RC; ++i)
    if (t + 256 * i < nf) put(t + 256 * i, keep[i], e);
  for (int c = t + 256 * RC; c < nf; c += 256) {
    Chunk d;
    float v[8];
    load(c, d);
    values(d, v);
    put(c, v, e);
  }
  if (t < Np - 8 * nf) {                         // the last elements and the zeros behind them
    const float x = ldexpf(rest, -e);
    const _Float16 h = (_Float16)x;
    const int at = 8 * nf + t;
    o[at] = __builtin_bit_cast(uint16_t, h);
    if constexpr (TERMS == 2) o[(size_t)M * Np + at] = __builtin_bit_cast(uint16_t, second_term(x, h));
  }
}

// ---- the GEMM ----------------------------------------------------------------------------------------------------
constexpr int kCols = 256;             // output columns of a tile
constexpr int kSlots = 512;            // workgroups the chip runs at once
constexpr int kScaleRow = 72;          // float16 scales of one group: 64 n, padded so that the 4 records' writes spread over the banks
constexpr int kABytes = 128 * 32;      // activation bytes per 32 rows and stage

// Formats: 0 FP8, 1 NVFP4, 2 and 3 AWQ with metadata layout 3 and 4.  NVFP4 has 16 rows of group scales per stage, AWQ 8 of
// scales and 8 of biases.
constexpr bool is_awq(int fmt) { return fmt >= 2; }
template <int FMT> constexpr int b_stage() { return FMT == 0 ? 64 * 256 : 64 * 128 + 16 * kScaleRow * 2; }
// The epilogue reuses the stages: 32 x 64 float32 per wave, rows padded by 16 bytes; the tile's row scales lie behind both.
constexpr int kEpiRow = 64 + 4, kEpiBytes = 32 * kEpiRow * 4;
template <int FMT> constexpr int grad_scale_at(int mb) {
  const int stages = 2 * (mb * kABytes + b_stage<FMT>());
  return stages > 4 * kEpiBytes ? stages : 4 * kEpiBytes;
}
template <int FMT> constexpr int grad_lds(int mb) { return grad_scale_at<FMT>(mb) + 128 * 4; }

// Work plan, a function of the shape: tiles of bm x 256, of which the last round may be cut into S parts of `per` steps of 64 n,
// whose float32 sums a second kernel adds in order.
struct GradPlan {
  int mb, bm, ntm, ntk, tiles, steps;  // mb: activation blocks of 32 rows (of one term) per tile
  int full, S, per, units;             // tiles [0, full) run whole; units = (tiles - full) * S parts
};
// The plan is the one of least estimated time, in us: a step of a 128-row tile takes 0.55 us of its CU (a quarter of that does not
// shrink with the rows: weights and their decoding) and never less than 0.9 (a copy's way through memory); a tile's rows take 1.2
// per 32 of them to leave; split tiles write and read their sums at 4.5 TB/s and take a further launch of 2.5.  At 512 x 1024 -> 8192 four parts per tile cost 35 us and whole
// tiles 17; at 512 x 17408 -> 5120 six parts take 98 us and whole tiles, on 80 of 256 CUs, 190.
inline GradPlan grad_plan(int M, int N, int K, int terms) {
  GradPlan best{};
  double least = 1e30;
  for (int mb = 4; mb >= terms; mb /= 2) {
    GradPlan p{};
    p.mb = mb;
    p.bm = 32 * mb / terms;
    if (mb > terms && M <= p.bm / 2) continue;   // half the tile would stay empty
    p.ntm = (M + p.bm - 1) / p.bm;
    p.ntk = (K + kCols - 1) / kCols;
    p.tiles = p.ntm * p.ntk;
    p.steps = (N + 63) / 64;
    auto step_us = [&](int64_t wgs) {            // of one workgroup, with wgs of them (at most two per CU at once) on the chip
      const double share = (double)std::min<int64_t>(2, (wgs + 255) / 256);
      return std::max(0.9, 0.55 * share * (0.25 + 0.1875 * mb));
    };
    for (int split = 0; split < 2; ++split) {    // whole tiles only, or the last round in parts
      const int tail = split ? p.tiles % kSlots : 0;
      if (split && tail == 0) continue;
      const int full = p.tiles - tail;
      const double body = full == 0 ? 0 : (double)((full + kSlots - 1) / kSlots) * (p.steps * step_us(full) + 1.2 * mb);
      const int most = split ? std::min(p.steps, std::max(1, kSlots / tail)) : 1;
      for (int s = split ? 2 : 1; s <= most; ++s) {
        GradPlan q = p;
        q.full = full;
        q.per = (p.steps + s - 1) / s;
        q.S = split ? (p.steps + q.per - 1) / q.per : 1;
        q.units = tail * q.S;
        const double bytes = (double)q.units * p.bm * kCols * 4;
        if (bytes > (double)((size_t)64 << 20)) break;
        const double us = body + (split ? q.per * step_us(q.units) + 1.2 * mb + 2.5 + bytes * 2 / 4.5e6 : 0.0);
        if (us < least) least = us, best = q;
      }
    }
  }
  return best;
}

typedef __attribute__((address_space(3))) const uint8_t lds_u8;
typedef int i32x2 __attribute__((ext_vector_type(2)));

template <int FMT, int MB, int TERMS>
__global__ void __launch_bounds__(256, 2) grad_gemm_kernel(int M, int N, int Np, int K, GradPlan plan,
                                                           const uint16_t* __restrict__ a16,
                                                           const float* __restrict__ rowscale,
                                                           const uint8_t* __restrict__ w, AwqLayout L, float inv,
                                                           void* __restrict__ dx, bool dx_bf, float* __restrict__ partials) {
  constexpr int RB = MB / TERMS;               // 32-row blocks of the output tile
  constexpr int BM = 32 * RB;
  constexpr int ASTAGE = MB * kABytes, BSTAGE = b_stage<FMT>(), STAGE = ASTAGE + BSTAGE;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 31, h = lane >> 5;

  // Parts of the split tiles first, then whole tiles: workgroup b runs on XCD b % 8, and each XCD gets a contiguous
  // run of tiles, ordered in bands of 8 tile rows so that the tiles in flight share rows and columns in its L2.
  const int b = (int)blockIdx.x;
  const int ugrid = (plan.units + 7) & ~7;
  int tile, part = -1, s0 = 0, s1 = plan.steps;
  if (b < ugrid) {
    if (b >= plan.units) return;
    tile = plan.full + b / plan.S;
    part = b % plan.S;
    s0 = part * plan.per;
    s1 = min(s0 + plan.per, plan.steps);
  } else {
    const int f = b - ugrid, per = ((int)gridDim.x - ugrid) >> 3;
    tile = (f & 7) * per + (f >> 3);
    if (tile >= plan.full) return;
  }
  const int band = tile / (8 * plan.ntk), in = tile - band * 8 * plan.ntk;
  const int height = min(8, plan.ntm - 8 * band);
  const int tm = 8 * band + in % height, tk = in / height;
  const int m0 = tm * BM, k0 = tk * kCols;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  // Activation copies: a wave moves rows 8 MB wave .. + 8 MB - 1 of the MB * 32 LDS rows (row r of term t is LDS row
  // 32 RB t + r), 8 rows per copy; 16-byte chunk c of a row is stored at c ^ ((row >> 1) & 7), which spreads the
  // fragment reads of 16 rows over all 64 banks.
  uint32_t aoff[MB];
  const uint8_t* abase[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int p = 64 * MB * wave + 64 * i + lane, row = p >> 3, c = p & 7;
    const int t = __builtin_amdgcn_readfirstlane((8 * MB * wave + 8 * i) / BM);   // the term: 8 rows never straddle one
    const int r = row - t * BM;
    abase[i] = reinterpret_cast<const uint8_t*>(a16) + ((size_t)t * M + m0) * (size_t)Np * 2;
    aoff[i] = (uint32_t)(min(m0 + r, M - 1) - m0) * (uint32_t)Np * 2u + (uint32_t)((c ^ ((row >> 1) & 7)) * 16);
  }
  auto copy_a = [&](int step, int stage) {
    const uint32_t sb = __builtin_amdgcn_readfirstlane(lds0 + stage * STAGE + 1024 * MB * wave);
    const uint8_t* bases[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) bases[i] = abase[i] + (size_t)step * 128 - 1024 * i;
    lds_copy16_run<MB>(aoff, bases, sb);
  };

  // FP8 weight copies: rows of 256 bytes, 16 rows per wave, 4 rows per copy; chunk c of row r at c ^ (r & 15).  Rows
  // past N and columns past K repeat the last ones (their products meet zeros of dy or are not stored).
  const int rb = FMT == 0 ? K : (FMT == 1 ? (K >> 6) * 36 : K >> 1);   // bytes of a weight row
  uint32_t woff[4];
  // NVFP4: thread t loads record t % 4 of row t / 4 of a step into registers and writes it to LDS a step later.
  const uint8_t* nvbase = nullptr;
  if constexpr (FMT == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * wave + 4 * i + (lane >> 4), c = (lane & 15) ^ (r & 15);
      woff[i] = (uint32_t)min(16 * c, K - 16 - k0);
    }
  } else if constexpr (FMT == 1) {
    nvbase = w + (size_t)min((k0 >> 6) + (tid & 3), (K >> 6) - 1) * 36;
  }
  auto copy_w = [&](int step, int stage) {          // FP8
    const uint32_t sb = __builtin_amdgcn_readfirstlane(lds0 + stage * STAGE + ASTAGE + 4096 * wave);
    const int n0 = 64 * step + 16 * wave;
    const int nb = min(n0, N - 1);
    const uint8_t* base = w + (size_t)nb * rb + k0;
    uint32_t v[4];
    const uint8_t* bases[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = min(n0 + 4 * i + (lane >> 4), N - 1);
      v[i] = (uint32_t)(n - nb) * (uint32_t)rb + woff[i];
      bases[i] = base - 1024 * i;
    }
    lds_copy16_run<4>(v, bases, sb);
  };
  struct Rec { u32x3_a4 a, b, c; };                  // 36 bytes: scale dword, 8 nibble dwords
  struct AwqRec { u32x4 c[2]; uint32_t s[2], z[2]; };  // two groups of a row: codes, scales, zeros or biases
  std::conditional_t<is_awq(FMT), AwqRec, Rec> rec;
  // AWQ: thread t loads groups 2 (t % 4) and the next of row t / 4 of a step (past K the last one again, not stored)
  const int g0 = min((k0 >> 5) + 2 * (tid & 3), (int)L.G - 1), g1 = min(g0 + 1, (int)L.G - 1);
  auto load_rec = [&](int step) {                    // NVFP4, AWQ
    const size_t n = (size_t)min(64 * step + (tid >> 2), N - 1);
    if constexpr (is_awq(FMT)) {
      const size_t at = n * (size_t)L.G;
      const uint16_t* sc = reinterpret_cast<const uint16_t*>(w + L.scale_off) + at;
      rec.c[0] = *reinterpret_cast<const u32x4*>(w + n * rb + 16 * g0);
      rec.c[1] = *reinterpret_cast<const u32x4*>(w + n * rb + 16 * g1);
      rec.s[0] = sc[g0];
      rec.s[1] = sc[g1];
      if constexpr (FMT == 2) {
        const uint8_t* z = w + L.meta2_off + at;
        rec.z[0] = z[g0];
        rec.z[1] = z[g1];
      } else {
        const uint16_t* z = reinterpret_cast<const uint16_t*>(w + L.meta2_off) + at;
        rec.z[0] = z[g0];
        rec.z[1] = z[g1];
      }
    } else {
      const uint8_t* p = nvbase + n * rb;
      rec.a = *reinterpret_cast<const u32x3_a4*>(p);
      rec.b = *reinterpret_cast<const u32x3_a4*>(p + 12);
      rec.c = *reinterpret_cast<const u32x3_a4*>(p + 24);
    }
  };
  auto write_rec = [&](int stage) {
    uint8_t* bs = lds + stage * STAGE + ASTAGE;
    const int r = tid >> 2, q = tid & 3, sw = (r >> 1) & 7;
    if constexpr (is_awq(FMT)) {
      uint16_t* sc = reinterpret_cast<uint16_t*>(bs + 64 * 128) + 2 * q * kScaleRow + r;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<u32x4*>(bs + r * 128 + (((2 * q + j) ^ sw) * 16)) = rec.c[j];
        const _Float16 sv = f16_from_bits((uint16_t)rec.s[j]);
        sc[j * kScaleRow] = (uint16_t)rec.s[j];
        sc[(8 + j) * kScaleRow] = FMT == 2 ? __builtin_bit_cast(uint16_t, awq_bias(rec.z[j], sv)) : (uint16_t)rec.z[j];
      }
    } else {
      *reinterpret_cast<u32x4*>(bs + r * 128 + (((2 * q) ^ sw) * 16)) = u32x4{rec.a.y, rec.a.z, rec.b.x, rec.b.y};
      *reinterpret_cast<u32x4*>(bs + r * 128 + (((2 * q + 1) ^ sw) * 16)) = u32x4{rec.b.z, rec.c.x, rec.c.y, rec.c.z};
      const uint32_t d0 = as_u32(e4m3x2_f16<false>(rec.a.x)), d1 = as_u32(e4m3x2_f16<true>(rec.a.x));
      uint16_t* sc = reinterpret_cast<uint16_t*>(bs + 64 * 128) + 4 * q * kScaleRow + r;
      sc[0] = (uint16_t)d0;
      sc[kScaleRow] = (uint16_t)(d0 >> 16);
      sc[2 * kScaleRow] = (uint16_t)d1;
      sc[3 * kScaleRow] = (uint16_t)(d1 >> 16);
    }
  };

  f32x16 acc[MB][2];                         // block i: rows 32 (i % RB) .. of the tile, term i / RB
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // Fragments of sub-step s (16 n): activations chunk 2 s + h of each row; weights raw, 8 bytes along n per column.
  struct Raw { i32x2 q[FMT == 0 ? 2 : 1]; u32x4 d, z; };
  auto read_a = [&](int stage, int s, f16x8* af) {
    const uint8_t* ast = lds + stage * STAGE;
#pragma unroll
    for (int i = 0; i < MB; ++i)
      af[i] = *reinterpret_cast<const f16x8*>(ast + (32 * i + li) * 128 + (((2 * s + h) ^ ((li >> 1) & 7)) * 16));
  };
  // ds_read_b64_tr_b8: 16 lanes read 8 rows of 16 bytes, lanes 2j and 2j + 1 row j; lanes 0-15 and 16-31 take two
  // neighbouring chunks of rows 8h .. 8h + 7 of the sub-step, h = lane / 32.
  const int tr_row = 8 * h + ((lane & 15) >> 1), tr_half = (lane & 1) * 8, tr_chunk = (lane >> 4) & 1;
  auto read_b = [&](int stage, int s, Raw& raw) {
    lds_u8* bs = (lds_u8*)(lds + stage * STAGE + ASTAGE);
    const int r = 16 * s + tr_row;
    if constexpr (FMT == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = 4 * wave + 2 * j + tr_chunk;
        raw.q[j] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2*)(bs + r * 256 + ((c ^ (r & 15)) * 16) + tr_half));
      }
    } else {
      const int c = 2 * wave + tr_chunk;
      raw.q[0] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (__attribute__((address_space(3))) i32x2*)(bs + r * 128 + ((c ^ ((r >> 1) & 7)) * 16) + tr_half));
      // the lane's byte column li lies in group li / 8 of record `wave` (AWQ: in group 2 wave + li / 16); its 8 n
      const int group = is_awq(FMT) ? 2 * wave + (li >> 4) : 4 * wave + (li >> 3);
      const uint8_t* meta = lds + stage * STAGE + ASTAGE + 64 * 128 + (group * kScaleRow + 16 * s + 8 * h) * 2;
      raw.d = *reinterpret_cast<const u32x4*>(meta);
      if constexpr (is_awq(FMT)) raw.z = *reinterpret_cast<const u32x4*>(meta + 8 * kScaleRow * 2);
    }
  };
  auto decode = [&](const Raw& raw, f16x8* bf) {
    if constexpr (FMT == 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f16x2 p0 = e4m3x2_f16<false>(raw.q[j].x), p1 = e4m3x2_f16<true>(raw.q[j].x);
        const f16x2 p2 = e4m3x2_f16<false>(raw.q[j].y), p3 = e4m3x2_f16<true>(raw.q[j].y);
        bf[j] = f16x8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
      }
    } else if constexpr (is_awq(FMT)) {
      // low nibbles: even k, high nibbles: odd k; dword j holds 4 n
      f16x2 ev[4], od[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t wd = (uint32_t)(j ? raw.q[0].y : raw.q[0].x), lo = wd & 0x0F0F0F0Fu, hi = (wd >> 4) & 0x0F0F0F0Fu;
        const f16x2 s0 = as_f16x2(j ? raw.d.z : raw.d.x), s1 = as_f16x2(j ? raw.d.w : raw.d.y);
        const f16x2 z0 = as_f16x2(j ? raw.z.z : raw.z.x), z1 = as_f16x2(j ? raw.z.w : raw.z.y);
        ev[2 * j] = __builtin_elementwise_fma(nibbles_f16<false>(lo), s0, z0);
        ev[2 * j + 1] = __builtin_elementwise_fma(nibbles_f16<true>(lo), s1, z1);
        od[2 * j] = __builtin_elementwise_fma(nibbles_f16<false>(hi), s0, z0);
        od[2 * j + 1] = __builtin_elementwise_fma(nibbles_f16<true>(hi), s1, z1);
      }
      bf[0] = f16x8{ev[0].x, ev[0].y, ev[1].x, ev[1].y, ev[2].x, ev[2].y, ev[3].x, ev[3].y};
      bf[1] = f16x8{od[0].x, od[0].y, od[1].x, od[1].y, od[2].x, od[2].y, od[3].x, od[3].y};
    } else {
      // low nibbles: even k, high nibbles: odd k; the pairs (n, n + 1) of one k are put into one byte for the decoder
      const uint32_t wd[2] = {(uint32_t)raw.q[0].x, (uint32_t)raw.q[0].y};
      f16x2 ev[4], od[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t lo = (wd[j] & 0x000F000Fu) | ((wd[j] >> 4) & 0x00F000F0u);
        const uint32_t hi = ((wd[j] >> 4) & 0x000F000Fu) | ((wd[j] >> 8) & 0x00F000F0u);
        const f16x2 sa = as_f16x2(j ? raw.d.z : raw.d.x), sb = as_f16x2(j ? raw.d.w : raw.d.y);
        ev[2 * j] = e2m1x2_f16<0>(lo) * sa;
        ev[2 * j + 1] = e2m1x2_f16<2>(lo) * sb;
        od[2 * j] = e2m1x2_f16<0>(hi) * sa;
        od[2 * j + 1] = e2m1x2_f16<2>(hi) * sb;
      }
      bf[0] = f16x8{ev[0].x, ev[0].y, ev[1].x, ev[1].y, ev[2].x, ev[2].y, ev[3].x, ev[3].y};
      bf[1] = f16x8{od[0].x, od[0].y, od[1].x, od[1].y, od[2].x, od[2].y, od[3].x, od[3].y};
    }
  };
  auto mfmas = [&](const f16x8* af, const Raw& raw) {
    f16x8 bf[2];
    decode(raw, bf);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[i], bf[j], acc[i][j], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * MB; ++i) {       // one MFMA, one fragment read, two ALU operations at a time
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < MB + 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
    }
  };

  const int last = s1 - 1;
  auto fetch = [&](int step, int stage) {     // copies of a step
    copy_a(step, stage);
    if constexpr (FMT == 0) copy_w(step, stage);
  };
  // Prologue: steps s0 and s0 + 1 on their way, step s0 landed.  The tile's row scales come along for the epilogue.
  const float row_scale = tid < BM ? rowscale[min(m0 + tid, M - 1)] : 0.f;
  if constexpr (FMT != 0) load_rec(s0);
  fetch(s0, 0);
  if constexpr (FMT != 0) {
    write_rec(0);
    load_rec(min(s0 + 1, last));
  }
  if (s0 < last) fetch(s0 + 1, 1);
  // NVFP4: the records of step s0 have been waited for, and with them everything issued before; FP8: all but the second fetch
  if constexpr (FMT == 0) {
    if (s0 < last) wait_vmem<MB + 4>();
    else wait_vmem<0>();
  } else if constexpr (is_awq(FMT)) {
    // how many instructions a record's loads become is the compiler's choice: only the copies behind them stay out
    if (s0 < last) wait_vmem<MB>();
    else wait_vmem<0>();
  } else {
    if (s0 < last) wait_vmem<MB + 3>();
    else wait_vmem<3>();
  }
  wait_lds();
  __syncthreads();
  f16x8 af0[MB], af1[MB];
  Raw raw0, raw1;
  read_a(0, 0, af0);
  read_b(0, 0, raw0);
  for (int s = s0; s < s1; ++s) {
    const int st = (s - s0) & 1;
    read_a(st, 1, af1);
    read_b(st, 1, raw1);
    mfmas(af0, raw0);
    __builtin_amdgcn_sched_barrier(0);
    read_a(st, 2, af0);
    read_b(st, 2, raw0);
    mfmas(af1, raw1);
    __builtin_amdgcn_sched_barrier(0);
    read_a(st, 3, af1);
    read_b(st, 3, raw1);
    mfmas(af0, raw0);
    __builtin_amdgcn_sched_barrier(0);
    // NVFP4: records of step s + 1 (its stage's last readers passed the previous barrier)
    if constexpr (FMT != 0) write_rec(st ^ 1);
    wait_vmem<0>();                            // step s + 1's copies (issued a step ago) landed
    wait_lds();                                // this wave's reads of stage st are in registers, its writes in LDS
    __syncthreads();
    if constexpr (FMT != 0) load_rec(min(s + 2, last));
    if (s + 2 <= last) fetch(s + 2, st);
    read_a(st ^ 1, 0, af0);
    read_b(st ^ 1, 0, raw0);
    mfmas(af1, raw1);
    __builtin_amdgcn_sched_barrier(0);
  }
  // Epilogue, 32 rows at a time through LDS of the wave's own (every wave is done with the stages), so that rows leave in 16-byte
  // pieces: stored from the MFMA layout, element by element with its own address, a 128-row tile took 6 us by itself.
  const float rsc = row_scale;
  float* rscale = reinterpret_cast<float*>(lds + grad_scale_at<FMT>(MB));
  if (tid < BM) rscale[tid] = rsc;
  __syncthreads();
  float* ep = reinterpret_cast<float*>(lds + wave * kEpiBytes);
  const float c = FMT == 0 ? 1.0f : inv;
  if constexpr (TERMS == 2) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(acc[i + RB][j][r], 1.0f / kSecond, acc[i][j][r]);
  }
  float* pt = partials + (size_t)b * BM * kCols + 64 * wave;            // split tile: raw sums [BM][256] for grad_finish_kernel
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    wave_lds_fence();
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float* e = ep + (8 * (r >> 2) + 4 * h + (r & 3)) * kEpiRow;
      if constexpr (FMT == 0) {
        e[li] = acc[i][0][r];
        e[32 + li] = acc[i][1][r];
      } else {
        *reinterpret_cast<f32x2*>(e + 2 * li) = f32x2{acc[i][0][r], acc[i][1][r]};
      }
    }
    wave_lds_fence();
    if (part < 0 && dx_bf) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int p = lane + 64 * q, row = 32 * i + (p >> 3), col = 8 * (p & 7), m = m0 + row, k = k0 + 64 * wave + col;
        const float* e = ep + (p >> 3) * kEpiRow + col;
        const f32x4 u = *reinterpret_cast<const f32x4*>(e), v = *reinterpret_cast<const f32x4*>(e + 4);
        const float rs = rscale[row];
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = (j < 2 ? u[2 * j] : v[2 * j - 4]) * c * rs, x1 = (j < 2 ? u[2 * j + 1] : v[2 * j - 3]) * c * rs;
          o[j] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x0) | ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x1) << 16);
        }
        if (m < M && k < K)
          *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(dx) + (size_t)m * K + k) = u32x4{o[0], o[1], o[2], o[3]};
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int p = lane + 64 * q, row = 32 * i + (p >> 4), col = 4 * (p & 15), m = m0 + row, k = k0 + 64 * wave + col;
        const f32x4 v = *reinterpret_cast<const f32x4*>(ep + (p >> 4) * kEpiRow + col);
        if (part >= 0) {
          if (m < M) *reinterpret_cast<f32x4*>(pt + row * kCols + col) = v;
        } else if (m < M && k < K) {
          const float rs = rscale[row];
          *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(dx) + (size_t)m * K + k) =
              f32x4{v[0] * c * rs, v[1] * c * rs, v[2] * c * rs, v[3] * c * rs};
        }
      }
    }
  }
}

// dx of the split tiles: the S parts of every element added in order.  A thread takes 4 columns (K is a multiple
// of 16), a workgroup 4 rows of a tile.
__global__ void __launch_bounds__(256) grad_finish_kernel(int M, int K, GradPlan plan, const float* __restrict__ partials,
                                                          const float* __restrict__ rowscale, float c, void* __restrict__ dx,
                                                          bool dx_bf) {
  const int per_tile = plan.bm / 4;
  const int i = (int)blockIdx.x / per_tile, row = ((int)blockIdx.x - i * per_tile) * 4 + (int)(threadIdx.x >> 6);
  const int tile = plan.full + i;
  const int band = tile / (8 * plan.ntk), in = tile - band * 8 * plan.ntk;
  const int height = min(8, plan.ntm - 8 * band);
  const int tm = 8 * band + in % height, tk = in / height;
  const int m = tm * plan.bm + row, col = 4 * (int)(threadIdx.x & 63), k = tk * kCols + col;
  if (m >= M || k >= K) return;
  const size_t pt = (size_t)plan.bm * kCols;
  const float* p = partials + (size_t)i * plan.S * pt + row * kCols + col;
  f32x4 v = *reinterpret_cast<const f32x4*>(p);
  for (int s = 1; s < plan.S; ++s) v += *reinterpret_cast<const f32x4*>(p + s * pt);
  const float rs = rowscale[m];
  const size_t o = (size_t)m * K + k;
  float u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = v[j] * c * rs;
  if (dx_bf) {
    uint32_t hh[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) hh[j] = __builtin_bit_cast(uint16_t, (__bf16)u[j]);
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(dx) + o) = u32x2{hh[0] | (hh[1] << 16), hh[2] | (hh[3] << 16)};
  } else {
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(dx) + o) = f32x4{u[0], u[1], u[2], u[3]};
  }
}

inline int terms_of(XType dxt) { return dxt == X_F32 ? 2 : 1; }
// Workspace: float16 terms [TERMS][M][Np], row scales [M], split tiles' sums.
struct GradWs {
  size_t rs, partials, total;
};
inline GradWs grad_ws(int M, int N, int K, int terms) {
  const GradPlan p = grad_plan(M, N, K, terms);
  GradWs w;
  w.rs = align256((size_t)terms * M * p.steps * 64 * 2);
  w.partials = w.rs + align256((size_t)M * 4);
  w.total = w.partials + align256((size_t)p.units * p.bm * kCols * 4);
  return w;
}

template <int FMT, int MB, int TERMS>
hipError_t grad_gemm(int M, int N, int K, const GradPlan& p, const uint16_t* a16, const float* rs, const uint8_t* w,
                     const AwqLayout& L, float inv, void* dx, bool bf, float* partials, hipStream_t st) {
  if (!raise_lds_limit<grad_gemm_kernel<FMT, MB, TERMS>>()) return hipErrorInvalidValue;
  const int grid = ((p.units + 7) & ~7) + (p.full + 7) / 8 * 8;
  hipLaunchKernelGGL((grad_gemm_kernel<FMT, MB, TERMS>), dim3(grid), dim3(256), grad_lds<FMT>(MB), st, M, N, p.steps * 64, K,
                     p, a16, rs, w, L, inv, dx, bf, partials);
  return hipGetLastError();
}

template <int FMT>
hipError_t grad_dispatch(int M, int N, int K, int terms, const GradPlan& p, const uint16_t* a16, const float* rs,
                         const uint8_t* w, const AwqLayout& L, float inv, void* dx, bool bf, float* partials, hipStream_t st) {
  const int mb = p.mb;
  if (terms == 2)
    return mb == 2 ? grad_gemm<FMT, 2, 2>(M, N, K, p, a16, rs, w, L, inv, dx, bf, partials, st)
                   : grad_gemm<FMT, 4, 2>(M, N, K, p, a16, rs, w, L, inv, dx, bf, partials, st);
  if (mb == 1) return grad_gemm<FMT, 1, 1>(M, N, K, p, a16, rs, w, L, inv, dx, bf, partials, st);
  if (mb == 2) return grad_gemm<FMT, 2, 1>(M, N, K, p, a16, rs, w, L, inv, dx, bf, partials, st);
  return grad_gemm<FMT, 4, 1>(M, N, K, p, a16, rs, w, L, inv, dx, bf, partials, st);
}

// 3 register chunks cover rows of 6144, 9 rows of 18432.
template <bool BF, bool SC, int TERMS>
void grad_prep(int M, int N, int Np, const void* dy, const float* scale, uint16_t* a16, float* rs, hipStream_t st) {
  if (Np <= 3 * 2048)
    hipLaunchKernelGGL((grad_prep_kernel<BF, SC, TERMS, 3>), dim3(M), dim3(256), 0, st, M, N, Np, dy, scale, a16, rs);
  else
    hipLaunchKernelGGL((grad_prep_kernel<BF, SC, TERMS, 9>), dim3(M), dim3(256), 0, st, M, N, Np, dy, scale, a16, rs);
}
template <bool BF, bool SC, typename... A>
void grad_prep_terms(int terms, A... a) {
  if (terms == 2) grad_prep<BF, SC, 2>(a...);
  else grad_prep<BF, SC, 1>(a...);
}

}  // namespace

size_t linear_grad_scratch_bytes(int fmt, int M, int N, int K, XType dxt) {
  return grad_ws(M, N, K, terms_of(dxt)).total;
}

namespace {

hipError_t linear_grad(int fmt, int terms, int M, int N, int K, const void* dy, XType dyt, const uint8_t* w, const float* scale,
                       const AwqLayout& L, float inv, void* ws, void* dx, XType dxt, hipStream_t st) {
  const GradPlan p = grad_plan(M, N, K, terms);
  const GradWs W = grad_ws(M, N, K, terms);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  uint16_t* a16 = reinterpret_cast<uint16_t*>(base);
  float* rs = reinterpret_cast<float*>(base + W.rs);
  float* partials = reinterpret_cast<float*>(base + W.partials);
  const int Np = p.steps * 64;
  const bool bf = dxt == X_BF16;
  if (dyt == X_BF16) {
    if (fmt == 0) grad_prep_terms<true, true>(terms, M, N, Np, dy, scale, a16, rs, st);
    else grad_prep_terms<true, false>(terms, M, N, Np, dy, scale, a16, rs, st);
  } else {
    if (fmt == 0) grad_prep_terms<false, true>(terms, M, N, Np, dy, scale, a16, rs, st);
    else grad_prep_terms<false, false>(terms, M, N, Np, dy, scale, a16, rs, st);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  switch (fmt) {
    case 0: e = grad_dispatch<0>(M, N, K, terms, p, a16, rs, w, L, inv, dx, bf, partials, st); break;
    case 1: e = grad_dispatch<1>(M, N, K, terms, p, a16, rs, w, L, inv, dx, bf, partials, st); break;
    case 2: e = grad_dispatch<2>(M, N, K, terms, p, a16, rs, w, L, inv, dx, bf, partials, st); break;
    default: e = grad_dispatch<3>(M, N, K, terms, p, a16, rs, w, L, inv, dx, bf, partials, st); break;
  }
  if (e != hipSuccess || p.units == 0) return e;
  hipLaunchKernelGGL(grad_finish_kernel, dim3((unsigned)(p.tiles - p.full) * (p.bm / 4)), dim3(256), 0, st, M, K, p,
                     partials, rs, fmt == 0 ? 1.0f : inv, dx, bf);
  return hipGetLastError();
}

// bfloat16 dy fits into one float16 term after the scaling, whatever dx's type.
inline int awq_grad_terms(XType dyt, XType dxt) { return dyt == X_F32 && dxt == X_F32 ? 2 : 1; }

}  // namespace

hipError_t launch_linear_grad(int fmt, int M, int N, int K, const void* dy, XType dyt, const uint8_t* w, const float* scale,
                              float inv, void* ws, void* dx, XType dxt, hipStream_t st) {
  return linear_grad(fmt, terms_of(dxt), M, N, K, dy, dyt, w, scale, AwqLayout{}, inv, ws, dx, dxt, st);
}

size_t awq_linear_grad_scratch_bytes(int M, int N, int K, XType dyt, XType dxt) {
  return M == 0 ? 0 : grad_ws(M, N, K, awq_grad_terms(dyt, dxt)).total;
}

hipError_t launch_awq_linear_grad(int M, int N, int K, const void* dy, XType dyt, const uint8_t* bank, int meta_layout, void* ws,
                                  void* dx, XType dxt, hipStream_t st) {
  return linear_grad(meta_layout == 3 ? 2 : 3, awq_grad_terms(dyt, dxt), M, N, K, dy, dyt, bank, nullptr,
                     awq_layout(N, K, meta_layout), 1.f, ws, dx, dxt, st);
}

}  // namespace wq
