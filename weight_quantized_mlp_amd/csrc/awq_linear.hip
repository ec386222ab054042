// Linear with AWQ int4 group-32 weights (gfx950): awq_linear_run in include/wqmlp_blocks.h,
//   y[m,n] = sum_k x[m,k] dq[n,k],  dq = RN_f16(q scale + bias) exactly as the routed step decodes it.
//
// The weights are decoded in registers, straight from the packed bytes, into matrix-core operands (awq_common.h); x is
// turned into float16 terms (awq_pack_kernel), in the order the matrix cores read it.
//   Up to kOwnRows rows (awq_rows_kernel) and up to kFewRows (awq_shared_kernel): the weights' bytes bound it, and with them the
//     decode, so what matters is that every CU has work from the start and reads whole cache lines.  x is turned into terms by the
//     waves themselves, which spares a launch.  Calls in a row: 1 float16 row 5120 -> 17408 13-15 us (53 MB, 3.5-4.1 TB/s; bfloat16 16,
//     float32 18), 17408 -> 5120 17 (20.5, 23); 13 bfloat16 rows 17408 -> 5120 18-20 us, of which the parts' sum takes 4.
//   More rows (awq_gemm_kernel): the matrix cores bound it.  4 waves with 64 weight rows each share the tile of x through
//     LDS (global->LDS copies, two stages); every wave decodes only its own weights, once per tile row.  2049 bfloat16 rows
//     5120 -> 17408: 447 us (817 TFLOP/s), of which x's terms take 15 and the cut tiles' sum 15; a float16 product of those sizes in
//     the library 409.  512 rows: 147 us; 2048 float32 rows 17408 -> 5120, twice the products: 792-836.
// All split the contraction over workgroups where there are few; a further kernel adds the parts in order.
#include <algorithm>

#include "awq_common.h"
#include "dev_common.h"
#include "launch.h"

namespace wq {

namespace {

// ---- x -> float16 terms in fragment order ------------------------------------------------------------------------
// xp[m / 16][step][term][i][lane][8]: lane = 16 * quarter + m % 16 holds octet i of group 4 step + quarter of row m.
// Zeros past K (up to `steps`) and past M (up to a whole 16 rows).
__device__ __forceinline__ size_t frag_at(int mt, int steps, int step, int terms, int term, int i, int lane) {
  return (((((size_t)mt * steps + step) * terms + term) * 4 + i) * 64 + lane) * 16;
}

// One workgroup per row.  Rows of the same 16 share cache lines of xp, so they go to one XCD (workgroup b runs on XCD b % 8).
template <int XT, int TERMS>
__global__ void __launch_bounds__(256) awq_pack_kernel(int M, int K, int steps, const void* __restrict__ x, uint8_t* __restrict__ xp,
                                                       float* __restrict__ rowscale) {
  __shared__ float wmax[4];
  const int b = (int)blockIdx.x, t = (int)threadIdx.x;
  const int m = ((b >> 7) * 8 + (b & 7)) * 16 + ((b >> 3) & 15);
  const int rows = (M + 15) / 16 * 16;
  if (m >= rows) return;
  const int octets = steps * 16, real = K / 8;
  int e = 0;
  if constexpr (XT != X_F16) {
    float amax = 0.f;
    if (m < M)
      for (int o = t; o < real; o += 256) {
        float v[8];
        load_octet<XT>(x, (size_t)m * K + 8 * (size_t)o, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(v[j]));
      }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    if ((t & 63) == 0) wmax[t >> 6] = amax;
    __syncthreads();
    e = f16_row_exp(fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])));
  }
  if (t == 0) rowscale[m] = ldexpf(1.f, e);
  for (int o = t; o < octets; o += 256) {
    u32x4 w[TERMS];
    if (m < M && o < real) {
      float v[8];
      load_octet<XT>(x, (size_t)m * K + 8 * (size_t)o, v);
      octet_terms<TERMS>(v, e, w);
    } else {
#pragma unroll
      for (int j = 0; j < TERMS; ++j) w[j] = u32x4{0, 0, 0, 0};
    }
    const int step = o >> 4, lane = ((o >> 2) & 3) * 16 + (m & 15);
#pragma unroll
    for (int j = 0; j < TERMS; ++j)
      *reinterpret_cast<u32x4*>(xp + frag_at(m >> 4, steps, step, TERMS, j, o & 3, lane)) = w[j];
  }
}

// 4 results of row m from column n on, as far as the row goes.
__device__ __forceinline__ void store_row4(float* y, int N, int m, int n, f32x4 v) {
  float* o = y + (size_t)m * N + n;
  if (n + 3 < N && (N & 3) == 0) {
    *reinterpret_cast<f32x4*>(o) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < N) o[j] = v[j];
  }
}

// ---- up to kOwnRows rows -----------------------------------------------------------------------------------------
// A workgroup has 16 weight rows; its waves take blocks of 4 steps (16 groups, 512 k) in turn, a block's 4 KB of codes in flight
// behind the products of the block before.  The 16 rows' scales and zeros are two contiguous pieces of memory, which the workgroup copies
// to LDS at its start: read by the waves block by block, 32 and 16 bytes of a row at a time, they cost half of the codes' time (1 row
// 5120 -> 17408: 16.2 us, without them 11.8).
constexpr int kBlockSteps = 4;
constexpr int kOwnRows = 2;                    // (4 rows 5120 -> 17408: 22.3 us here, 19.3 in awq_shared_kernel)
constexpr int kRowsGroups = 1024;              // groups of a row at most: 48 or 64 KB of metadata

struct RowsPlan {
  int blocks, per, waves;                      // blocks per part, waves per workgroup
};

// MR rows of x (of which M are there): a wave scales its own 512 k of a row by their own power of two, so that no wave waits for
// another before the sums meet.  Part blockIdx.y of the blocks.
template <int ML, int XS, int MR>
__global__ void __launch_bounds__(512) awq_rows_kernel(int M, int N, int K, RowsPlan p, const void* __restrict__ x,
                                                       const uint8_t* __restrict__ bank, AwqLayout L, float* __restrict__ y,
                                                       float* __restrict__ partials) {
  constexpr int TERMS = XS == X_F32 ? 2 : 1;
  constexpr int COLS = 16 + 4;                                  // floats of an LDS row of sums: n, padded
  // The rows' scales, their zeros or biases, each wave's terms [MR][TERMS][1 KB].  All make room for the sums [wave][m][COLS].
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), q = lane >> 4;
  const int n0 = (int)blockIdx.x * 16, G = (int)L.G, rows = min(16, N - n0), nrow = min(lane & 15, rows - 1);
  const int b0 = (int)blockIdx.y * p.per, b1 = min(b0 + p.per, p.blocks);
  const uint8_t* codes = bank + (size_t)n0 * (L.G * 16);        // (offsets from it fit 32 bits)
  const int crow = nrow * G * 16;
  constexpr int ZB = ML == 3 ? 1 : 2;                           // bytes of a zero or bias
  const int sc = (rows * G * 2 + 15) >> 4, zc = (rows * G * ZB + 15) >> 4;   // 16-byte pieces (the planes are padded to whole ones)
  uint8_t* own = lds + (sc + zc) * 16 + wave * (MR * TERMS * 1024);
  const uint8_t* xs = own + min(lane & 15, MR - 1) * (TERMS * 1024) + q * 64;

  struct Block {
    RawOctet<XS> x[MR];
    u32x4 c[4];
  };
  auto load = [&](int b, Block& d) {
    const int o = min(64 * b + lane, K / 8 - 1);
#pragma unroll
    for (int m = 0; m < MR; ++m)
      d.x[m] = load_raw<XS>(static_cast<const uint8_t*>(x) + (size_t)min(m, M - 1) * K * (XS == X_F32 ? 4 : 2), (uint32_t)(8 * o));
#pragma unroll
    for (int t = 0; t < 4; ++t) d.c[t] = *reinterpret_cast<const u32x4*>(codes + (uint32_t)(crow + 16 * min(16 * b + 4 * t + q, G - 1)));
  };
  Block u, v;
  int b = b0 + wave;
  {
    constexpr int UP = 4;                                       // pieces of a thread on their way at once
    const u32x4* gs = reinterpret_cast<const u32x4*>(bank + L.scale_off + (size_t)n0 * G * 2);
    const u32x4* gz = reinterpret_cast<const u32x4*>(bank + L.meta2_off + (size_t)n0 * G * ZB) - sc;
    const int T = 64 * p.waves, last = sc + zc - 1;
    u32x4 piece[UP];
    auto load4 = [&](int i0) {
#pragma unroll
      for (int k = 0; k < UP; ++k) {
        const int i = min(i0 + k * T, last);
        piece[k] = (i < sc ? gs : gz)[i];
      }
    };
    load4(tid);
    if (b < b1) load(b, u);
    for (int i0 = tid; i0 <= last; i0 += UP * T) {
      if (i0 != tid) load4(i0);
#pragma unroll
      for (int k = 0; k < UP; ++k)
        if (i0 + k * T <= last) reinterpret_cast<u32x4*>(lds)[i0 + k * T] = piece[k];
    }
    __syncthreads();
  }

  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const uint8_t* smeta = lds + nrow * G * 2;
  const uint8_t* zmeta = lds + sc * 16 + nrow * G * ZB;
  auto multiply = [&](int b, const Block& d) {
    float scale[MR];
    wave_lds_fence();                                           // the last block's fragments are in registers
#pragma unroll
    for (int m = 0; m < MR; ++m) {                              // the wave's 64 octets of each row -> terms in its LDS
      u32x4 t[TERMS];
      scale[m] = wave_terms<XS, TERMS>(d.x[m], 64 * b + lane < K / 8, t);
#pragma unroll
      for (int j = 0; j < TERMS; ++j) *reinterpret_cast<u32x4*>(own + (m * TERMS + j) * 1024 + lane * 16) = t[j];
    }
    wave_lds_fence();
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int g = 16 * b + 4 * t + q, gc = min(g, G - 1);
      AwqStep a;
      a.s = *reinterpret_cast<const uint16_t*>(smeta + 2 * gc);
      if constexpr (ML == 3) a.z = zmeta[gc];
      else a.z = *reinterpret_cast<const uint16_t*>(zmeta + 2 * gc);
      f16x2 s2, b2;
      awq_meta<ML>(a, g < G, s2, b2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f16x8 w = awq_frag(d.c[t][i], s2, b2);
#pragma unroll
        for (int j = 0; j < TERMS; ++j)
          sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, *reinterpret_cast<const f16x8*>(xs + j * 1024 + t * 256 + i * 16), sum, 0, 0, 0);
      }
    }
    float rs = scale[0];                                        // of the lane's column: row lane % 16 of x
#pragma unroll
    for (int m = 1; m < MR; ++m) rs = (lane & 15) >= m ? scale[m] : rs;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = fmaf(sum[j], rs, acc[j]);
  };
  const int w = p.waves;
  if constexpr (MR == 1) {
    // Every path knows what it has on its way: behind a branch that the products after it share, they would wait for the next block's
    // loads, too (1 row 17408 -> 5120: 18.8 us, so 17.7; 2 float32 rows would lose a wave per SIMD to the copies: 27.8, 32.8).
    for (; b + w < b1; b += 2 * w) {
      load(b + w, v);
      __builtin_amdgcn_sched_barrier(0);
      multiply(b, u);
      if (b + 2 * w >= b1) {
        multiply(b + w, v);
        b = b1;
        break;
      }
      load(b + 2 * w, u);
      __builtin_amdgcn_sched_barrier(0);
      multiply(b + w, v);
    }
    if (b < b1) multiply(b, u);
  } else {
    for (; b < b1; b += 2 * w) {                                // (a load too many costs as much as one that is needed)
      if (b + w < b1) load(b + w, v);
      multiply(b, u);
      if (b + w >= b1) break;
      if (b + 2 * w < b1) load(b + 2 * w, u);
      multiply(b + w, v);
    }
  }

  // the waves' sums, in order
  __syncthreads();                                              // every wave is done with the metadata and its terms
  float* part = reinterpret_cast<float*>(lds);
  if ((lane & 15) < M) *reinterpret_cast<f32x4*>(part + (wave * M + (lane & 15)) * COLS + 4 * q) = acc;
  __syncthreads();
  for (int i = tid; i < M * 16; i += 64 * p.waves) {
    const int m = i >> 4, n = n0 + (i & 15);
    if (n >= N) continue;
    float r = 0.f;
    for (int k = 0; k < p.waves; ++k) r += part[(k * M + m) * COLS + (i & 15)];
    if (partials != nullptr) partials[((size_t)blockIdx.y * M + m) * N + n] = r;
    else y[(size_t)m * N + n] = r;
  }
}

// ---- up to kFewRows rows -----------------------------------------------------------------------------------------
// 8 waves with 16 weight rows each share x: CT tiles of 16 rows, SB blocks at a time, turned into terms in LDS once for 128 weight
// rows.  The contraction is split over workgroups until they fill the chip.  A row's metadata of SB blocks is 32 SB + 16 SB
// bytes, read whole into the wave's own LDS: with the codes of all SB blocks and x on their way at once, a pass has one memory latency.
constexpr int kFewRows = 32;
constexpr int kSharedWaves = 8;
// Blocks at a time for that many column tiles and terms: x and metadata leave room for two workgroups on a CU or more.
constexpr int shared_blocks(int tiles) { return tiles == 1 ? 2 : 1; }

template <int ML, int XS, int CT>
__global__ void __launch_bounds__(512, 4) awq_shared_kernel(int M, int N, int K, int passes, int per, const void* __restrict__ x,
                                                            const uint8_t* __restrict__ bank, AwqLayout L, float* __restrict__ y,
                                                            float* __restrict__ partials) {
  constexpr int TERMS = XS == X_F32 ? 2 : 1, SB = shared_blocks(CT * TERMS), ROW = SB * 1024 + 16;   // bytes of a staged row and term
  constexpr int ZB = ML == 3 ? 1 : 2, SROW = SB * 32, ZROW = SB * 16 * ZB, WMETA = 16 * (SROW + ZROW);
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];   // x [16 CT][TERMS][ROW], the waves' metadata, row scales
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), q = lane >> 4;
  const int n0 = ((int)blockIdx.x * kSharedWaves + wave) * 16, G = (int)L.G, octets = K / 8;
  uint8_t* smeta = lds + 16 * CT * TERMS * ROW + wave * WMETA;
  uint8_t* zmeta = smeta + 16 * SROW;
  float* scales = reinterpret_cast<float*>(lds + 16 * CT * TERMS * ROW + kSharedWaves * WMETA);
  const int p0 = (int)blockIdx.y * per, p1 = min(p0 + per, passes);
  // The last piece of the second plane starts here; a wave with rows whose pieces would reach further reads those one by one.
  // Offsets from the wave's first row (or the last one there is) fit 32 bits: 16 rows of at most 4 MB.
  const bool live_tile = n0 < N;
  const int base = min(n0, N - 1), top = N - 1 - base;          // rows from `base` on: at most `top`
  const int64_t zbytes = ZB * (int64_t)N * G, zat = (int64_t)base * G * ZB;
  const int zlast = (int)min((zbytes + 15) / 16 * 16 - 16 - zat, (int64_t)1 << 30);
  const uint8_t* codes = bank + (size_t)base * (L.G * 16);
  const uint8_t* splane = bank + L.scale_off + (size_t)base * G * 2;
  const uint8_t* zplane = bank + L.meta2_off + zat;
  const int crow = min(lane & 15, top) * G * 16;
  f32x4 acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int p = p0; p < p1; ++p) {
    constexpr int XR = 2 * CT;                                  // rows of x of a wave
    const int b0 = p * SB;
    RawOctet<XS> xr[XR][SB];
#pragma unroll
    for (int r = 0; r < XR; ++r)
#pragma unroll
      for (int j = 0; j < SB; ++j)
        xr[r][j] = load_raw<XS>(static_cast<const uint8_t*>(x) + (size_t)min(wave + 8 * r, M - 1) * K * (XS == X_F32 ? 4 : 2),
                                (uint32_t)(8 * min(64 * (b0 + j) + lane, octets - 1)));
    constexpr int SP = 16 * SROW / 16, ZP = 16 * ZROW / 16, SN = (SP + 63) / 64, ZN = (ZP + 63) / 64;   // pieces of a wave, per lane
    typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
    u32x4 sp[SN], zp[ZN];
#pragma unroll
    for (int j = 0; j < SN; ++j) {
      const int i = min(lane + 64 * j, SP - 1), r = i / (SROW / 16), c = i % (SROW / 16);
      sp[j] = *reinterpret_cast<const u32x4_a1*>(splane + (uint32_t)(2 * (min(r, top) * G + min(16 * b0 + 8 * c, G - 1))));
    }
#pragma unroll
    for (int j = 0; j < ZN; ++j) {
      const int i = min(lane + 64 * j, ZP - 1), r = i / (ZROW / 16), c = i % (ZROW / 16);
      zp[j] = *reinterpret_cast<const u32x4_a1*>(zplane + min(ZB * (min(r, top) * G + min(16 * b0 + (16 / ZB) * c, G - 1)), zlast));
    }
    u32x4 cd[SB][4];
#pragma unroll
    for (int j = 0; j < SB; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        cd[j][t] = *reinterpret_cast<const u32x4*>(codes + (uint32_t)(crow + 16 * min(16 * (b0 + j) + 4 * t + q, G - 1)));
    if (p != p0) __syncthreads();                               // the last pass's readers of x are done
#pragma unroll
    for (int r = 0; r < XR; ++r) {
      const int m = wave + 8 * r;
      if (m >= M) break;
      float amax = 0.f;
      if constexpr (XS != X_F16) {
#pragma unroll
        for (int j = 0; j < SB; ++j)
          if (64 * (b0 + j) + lane < octets) amax = fmaxf(amax, octet_max<XS>(xr[r][j]));
        amax = wave64_max(amax);
      }
      const int e = XS == X_F16 ? 0 : f16_row_exp(amax);
      if (lane == 0) scales[m] = ldexpf(1.f, e);
#pragma unroll
      for (int j = 0; j < SB; ++j) {
        u32x4 t[TERMS];
        raw_terms<XS, TERMS>(xr[r][j], e, 64 * (b0 + j) + lane < octets, t);
#pragma unroll
        for (int k = 0; k < TERMS; ++k) *reinterpret_cast<u32x4*>(lds + (m * TERMS + k) * ROW + (64 * j + lane) * 16) = t[k];
        __builtin_amdgcn_sched_barrier(0);                      // (interleaved, the octets' values spill)
      }
    }
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < SN; ++j)
      if (lane + 64 * j < SP) reinterpret_cast<u32x4*>(smeta)[lane + 64 * j] = sp[j];
#pragma unroll
    for (int j = 0; j < ZN; ++j)
      if (lane + 64 * j < ZP) reinterpret_cast<u32x4*>(zmeta)[lane + 64 * j] = zp[j];
    if (ZB * ((int64_t)min(15, top) * G + min(16 * (b0 + SB), G + 15)) > zlast) {
      wave_lds_fence();
      for (int i = lane; i < 16 * SB * 16; i += 64) {
        const int r = i / (SB * 16), g = i % (SB * 16);
        const int at = min(r, top) * G + min(16 * b0 + g, G - 1);
        if constexpr (ML == 3) zmeta[r * ZROW + g] = zplane[at];
        else *reinterpret_cast<uint16_t*>(zmeta + r * ZROW + 2 * g) = reinterpret_cast<const uint16_t*>(zplane)[at];
      }
    }
    __syncthreads();
    f32x4 sum[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) sum[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < SB; ++j) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int at = 16 * j + 4 * t + q;
        AwqStep a;
        a.s = *reinterpret_cast<const uint16_t*>(smeta + (lane & 15) * SROW + 2 * at);
        if constexpr (ML == 3) a.z = zmeta[(lane & 15) * ZROW + at];
        else a.z = *reinterpret_cast<const uint16_t*>(zmeta + (lane & 15) * ZROW + 2 * at);
        f16x2 s2, b2;
        awq_meta<ML>(a, 16 * b0 + at < G, s2, b2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f16x8 w = awq_frag(cd[j][t][i], s2, b2);
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const int m = min(16 * c + (lane & 15), M - 1);
#pragma unroll
            for (int k = 0; k < TERMS; ++k)
              sum[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                  w, *reinterpret_cast<const f16x8*>(lds + (m * TERMS + k) * ROW + (4 * at + i) * 16), sum[c], 0, 0, 0);
          }
        }
      }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const float rs = scales[min(16 * c + (lane & 15), M - 1)];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[c][j] = fmaf(sum[c][j], rs, acc[c][j]);
    }
  }
  if (!live_tile) return;
  float* out = partials != nullptr ? partials + (size_t)blockIdx.y * M * N : y;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int m = 16 * c + (lane & 15);
    if (m < M) store_row4(out, N, m, n0 + 4 * q, acc[c]);
  }
}

// ---- many rows ---------------------------------------------------------------------------------------------------
// Tile: 16 MT rows of x by 256 weight rows, 64 per wave.  Where the tiles of the last, unfilled round fit it twice or more, they are
// cut into S parts of `per` steps (bfloat16 rows 5120 -> 17408, uncut and cut: 48 99 and 48 us, 128 137 and 64, 256 138 and 96, 1024 297 and
// 232, 2049 469 and 447; 17408 -> 5120: 128 429 and 73, 512 434 and 148, 1024 463 and 245; cut tiles before the whole ones, which lets all
// run out of step and miss L2: 15% slower).  A last round of 257 to 511 tiles stays whole: 512 rows 5120 -> 17408 are 272, 148 us.
constexpr int kGemmCols = 256, kSlots = 512;   // workgroups the chip runs at once: two per CU

struct TilePlan {
  int mt, ntm, ntn, full, S, per, units, steps;   // tiles [0, full) run whole; units = the others' S parts
};
// Tile rows and columns of tile id: bands of 8 tile rows.
__device__ __forceinline__ void tile_of(const TilePlan& p, int id, int& tm, int& tn) {
  const int band = id / (8 * p.ntn), in = id - band * 8 * p.ntn, height = min(8, p.ntm - 8 * band);
  tm = 8 * band + in % height;
  tn = in / height;
}

template <int ML, int TERMS, int MT>
__global__ void __launch_bounds__(256, 2) awq_gemm_kernel(int M, int N, TilePlan p, const uint8_t* __restrict__ xp,
                                                          const float* __restrict__ rowscale, const uint8_t* __restrict__ bank,
                                                          AwqLayout L, float* __restrict__ y, float* __restrict__ partials) {
  constexpr int NT = 4, UNITS = MT * TERMS, STAGE = UNITS * 4096;   // a unit: one term of 16 rows, 4 KB per step
  constexpr int ZB = ML == 3 ? 1 : 2;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, G = (int)L.G;
  // Whole tiles first, then the others' parts.  Workgroup b runs on XCD b % 8: each XCD gets a contiguous run of either, so that those
  // in flight there share rows and weights in its L2, a tile's parts the lines of its scales and zeros (128 rows 5120 -> 17408: 63 us;
  // with the parts' tiles side by side 74).
  const int fgrid = (p.full + 7) & ~7;
  int b = (int)blockIdx.x, id, part = -1, s0 = 0, s1 = p.steps;
  if (b < fgrid) {
    id = (b & 7) * (fgrid >> 3) + (b >> 3);
    if (id >= p.full) return;
  } else {
    b -= fgrid;
    b = (b & 7) * (((int)gridDim.x - fgrid) >> 3) + (b >> 3);
    if (b >= p.units) return;
    const int tile = b / p.S;
    part = b - tile * p.S;
    id = p.full + tile;
    s0 = part * p.per;
    s1 = min(s0 + p.per, p.steps);
  }
  int tm, tn;
  tile_of(p, id, tm, tn);
  const int n0 = tn * kGemmCols + 64 * wave, mt0 = tm * MT, mtiles = (M + 15) >> 4;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  // Row tile r: rows first[r] .. + 15; past the matrix its last 16 again, of which only the rows not yet covered are stored.  Then a
  // lane's offset in every tile and step is the same, and the scalar bases do the rest.
  int first[NT];
#pragma unroll
  for (int r = 0; r < NT; ++r) first[r] = min(n0 + 16 * r, max(N - 16, 0));
  const int lrow = min(lane & 15, N - 1);
  const uint32_t coff = (uint32_t)(lrow * G * 16 + 16 * q), soff = (uint32_t)((lrow * G + q) * 2), zoff = (uint32_t)((lrow * G + q) * ZB);
  AwqStep wa[NT], wb[NT];
  auto load_w = [&](int step, AwqStep (&d)[NT]) {
    // the last step may have fewer than 4 groups: its lanes past the row's end read the row's last one
    const int back = max(4 * step + q - (G - 1), 0);
    const uint32_t co = coff - 16 * back, so = soff - 2 * back, zo = zoff - ZB * back;
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const size_t at = (size_t)first[r] * G + 4 * (size_t)step;
      d[r].c = *reinterpret_cast<const u32x4*>(bank + 16 * at + co);
      d[r].s = *reinterpret_cast<const uint16_t*>(bank + L.scale_off + 2 * at + so);
      if constexpr (ML == 3) d[r].z = *(bank + L.meta2_off + at + zo);
      else d[r].z = *reinterpret_cast<const uint16_t*>(bank + L.meta2_off + 2 * at + zo);
    }
  };
  // unit u = wave + 4 j: term u % TERMS of 16-row tile u / TERMS (past the end: the last one again, not stored)
  auto copy_x = [&](int step, int stage) {
#pragma unroll
    for (int j = 0; j < UNITS / 4; ++j) {
      const int u = wave + 4 * j, mt = min(mt0 + u / TERMS, mtiles - 1);
      const uint8_t* src = xp + frag_at(mt, p.steps, step, TERMS, u % TERMS, 0, 0);
      const uint8_t* bases[4] = {src, src, src, src};
      const uint32_t v = lane * 16, vs[4] = {v, v, v, v};
      lds_copy16_run<4>(vs, bases, __builtin_amdgcn_readfirstlane(lds0 + stage * STAGE + u * 4096));
    }
  };
  f32x4 acc[NT][MT];
#pragma unroll
  for (int r = 0; r < NT; ++r)
#pragma unroll
    for (int c = 0; c < MT; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Copies and weights are there.  (The uses of d are kept behind the wait: taken up into the step before, they would wait there.)
  auto landed = [&](AwqStep (&d)[NT]) {
    wait_vmem<0>();
#pragma unroll
    for (int r = 0; r < NT; ++r) asm volatile("" : "+v"(d[r].c), "+v"(d[r].s), "+v"(d[r].z));
  };
  // One step: the next one's weights and copies go out, this one's products, then the wait for both.
  auto step = [&](int s, int st, const AwqStep (&cur)[NT], AwqStep (&nxt)[NT]) {
    load_w(min(s + 1, s1 - 1), nxt);                    // (in the branch, the waits after it count for the worse of its sides)
    if (s + 1 < s1) copy_x(s + 1, st ^ 1);
    f16x2 s2[NT], b2[NT];
#pragma unroll
    for (int r = 0; r < NT; ++r) awq_meta<ML>(cur[r], 4 * s + q < G, s2[r], b2[r]);
    const uint8_t* xs = lds + st * STAGE + lane * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f16x8 w[NT];
#pragma unroll
      for (int r = 0; r < NT; ++r) w[r] = awq_frag(cur[r].c[i], s2[r], b2[r]);
#pragma unroll
      for (int c = 0; c < MT; ++c)
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          const f16x8 xf = *reinterpret_cast<const f16x8*>(xs + (c * TERMS + t) * 4096 + i * 1024);
#pragma unroll
          for (int r = 0; r < NT; ++r) acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[r], xf, acc[r][c], 0, 0, 0);
        }
    }
    // In order: 4 octets of x ahead of the products, each product followed by a share of the next weights' decode (2048 rows 5120 ->
    // 17408: 377 us, 381 as the compiler orders them; as two terms, 17408 -> 5120: 803 and 885; fewer rows lose by it).
    if constexpr (UNITS == 8) {
      __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 60, 0);
#pragma unroll
      for (int j = 0; j < 4 * UNITS; ++j) {
#pragma unroll
        for (int r = 0; r < NT; ++r) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (r == NT - 1 && j < 4 * UNITS - 4) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
        }
      }
    }
    landed(nxt);
    wait_lds();
    __syncthreads();
  };
  copy_x(s0, 0);
  load_w(s0, wa);
  landed(wa);
  __syncthreads();
  for (int s = s0; s < s1; s += 2) {
    step(s, 0, wa, wb);
    if (s + 1 < s1) step(s + 1, 1, wb, wa);
  }
  // Whole tiles: y.  Parts: [tile][part][16 MT][256], scaled, for awq_tiles_join_kernel.
  float* pt = part < 0 ? nullptr : partials + (size_t)b * (16 * MT * kGemmCols) + 64 * wave;
#pragma unroll
  for (int c = 0; c < MT; ++c) {
    const int ml = 16 * c + (lane & 15), m = 16 * mt0 + ml;
    if (m >= M) continue;
    const float rs = rowscale[m];
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const int n = first[r] + 4 * q, from = n0 + 16 * r;       // rows from `from` on are this tile's
      f32x4 v = acc[r][c];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= rs;
      if (part >= 0) {
        if (first[r] == from) *reinterpret_cast<f32x4*>(pt + ml * kGemmCols + 16 * r + 4 * q) = v;
        else
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j >= from && n + j < N) pt[ml * kGemmCols + n + j - n0] = v[j];
      } else if (first[r] == from) {
        store_row4(y, N, m, n, v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j >= from && n + j < N) y[(size_t)m * N + n + j] = v[j];
      }
    }
  }
}

// y of the cut tiles: a row of 256 columns per workgroup, the S parts in order.
__global__ void __launch_bounds__(256) awq_tiles_join_kernel(int M, int N, TilePlan p, const float* __restrict__ partials,
                                                             float* __restrict__ y) {
  const int rows = 16 * p.mt, i = (int)blockIdx.x / rows, ml = (int)blockIdx.x - i * rows;
  int tm, tn;
  tile_of(p, p.full + i, tm, tn);
  const int m = tm * rows + ml, n = tn * kGemmCols + (int)threadIdx.x;
  if (m >= M || n >= N) return;
  const size_t unit = (size_t)rows * kGemmCols;
  const float* f = partials + (size_t)i * p.S * unit + ml * kGemmCols + threadIdx.x;
  float v = f[0];
  for (int s = 1; s < p.S; ++s) v += f[s * unit];
  y[(size_t)m * N + n] = v;
}

// y = the sum of the S parts, in order.
__global__ void __launch_bounds__(256) awq_join_kernel(int M, int N, int S, const float* __restrict__ partials, float* __restrict__ y) {
  const int n = (int)blockIdx.x * 256 + (int)threadIdx.x, m = (int)blockIdx.y;
  if (n >= N) return;
  const size_t at = (size_t)m * N + n, part = (size_t)M * N;
  float v = 0.f;
  constexpr int UP = 16;                         // parts on their way at once
  for (int s0 = 0; s0 < S; s0 += UP) {
    float p[UP];
#pragma unroll
    for (int s = 0; s < UP; ++s)
      if (s0 + s < S) p[s] = partials[(s0 + s) * part + at];
#pragma unroll
    for (int s = 0; s < UP; ++s)
      if (s0 + s < S) v = s0 + s == 0 ? p[s] : v + p[s];
  }
  y[at] = v;
}

// ---- plan --------------------------------------------------------------------------------------------------------
// Workgroups of awq_shared_kernel to split up to: three per CU with two blocks at a time, else two.  256, 512, 768 and 1536 of them: 13
// bfloat16 rows 5120 -> 17408 24.5, 23.0, 19.1 and 19.1 us, 17408 -> 5120 20.7, 22.9, 19.6 and 19.5; 24 rows (one block at a time) 32.6, 23.9,
// 24.4 and 24.8, and 29.6, 23.3, 25.3 and 25.3; 8 float32 rows 28.0, 20.7, 20.8 and 20.1, and 25.8, 20.4, 21.2 and 21.4.  5120 -> 5120 and 2560 ->
// 9728, 4 to 24 rows: within 0.3 us of each other from 512 on.
constexpr int shared_fill(int tiles) { return tiles == 1 ? 768 : 512; }

struct AwqPlan {
  enum { kOwn, kShared, kTiles } kind;
  int terms, steps, S, per;    // S parts of `per` blocks (kOwn), passes (kShared) or steps (kTiles)
  int units;                   // blocks, passes
  int ct, waves;               // column tiles (kShared), waves (kOwn)
  TilePlan t;                  // kTiles
  size_t xp, rs, partials, total;
};
inline AwqPlan awq_plan(int M, int N, int K, XType xt) {
  AwqPlan p{};
  p.terms = awq_terms(xt);
  p.steps = (K + kStepK - 1) / kStepK;
  p.kind = M <= kOwnRows && K / 32 <= kRowsGroups ? AwqPlan::kOwn : (M <= kFewRows ? AwqPlan::kShared : AwqPlan::kTiles);
  const int64_t most = std::max<int64_t>(1, ((int64_t)64 << 20) / ((int64_t)M * N * 4));   // at most 64 MiB of parts
  const int blocks = (p.steps + kBlockSteps - 1) / kBlockSteps;
  if (p.kind == AwqPlan::kOwn) {
    p.units = blocks;
    const int64_t wgs = (N + 15) / 16;
    const int64_t S = std::min(std::max<int64_t>(1, std::min<int64_t>(256 / wgs, blocks / 12)), most);
    p.per = (int)((blocks + S - 1) / S);
    p.S = (blocks + p.per - 1) / p.per;
    // waves: at most 8, fewer where there are more workgroups than the chip then holds at once (20 waves per CU), and no more than the
    // number of turns needs; at least 4, which read the metadata.  5120 -> 17408, 1 row: 4 waves 14.3 us, 5 17.7, 8 17.2, 12 23;
    // 17408 -> 5120: 4 waves 17.4, 8 17.2, 12 19.7.
    int top = 8;
    while (top > 4 && wgs * p.S > 256 * (20 / top)) --top;
    const int turns = (p.per + top - 1) / top;
    p.waves = std::max(4, (p.per + turns - 1) / turns);
  } else if (p.kind == AwqPlan::kShared) {
    p.ct = M <= 16 ? 1 : 2;
    const int sb = shared_blocks(p.ct * p.terms), cols = (N + 16 * kSharedWaves - 1) / (16 * kSharedWaves);
    p.units = (blocks + sb - 1) / sb;
    const int64_t S = std::min(std::min<int64_t>(p.units, std::max(1, (shared_fill(p.ct * p.terms) + cols - 1) / cols)), most);
    p.per = (int)((p.units + S - 1) / S);
    p.S = (p.units + p.per - 1) / p.per;
  } else {
    TilePlan& t = p.t;
    t.mt = p.terms == 2 || M <= 64 ? 4 : 8;
    t.ntm = (M + 16 * t.mt - 1) / (16 * t.mt);
    t.ntn = (N + kGemmCols - 1) / kGemmCols;
    t.steps = p.steps;
    const int64_t tiles = (int64_t)t.ntm * t.ntn, tail = tiles % kSlots;
    const int64_t room = ((int64_t)64 << 20) / ((int64_t)16 * t.mt * kGemmCols * 4);       // parts in 64 MiB
    int64_t S = tail == 0 ? 1 : std::max<int64_t>(1, std::min<int64_t>({kSlots / tail, p.steps / 4, room / tail}));
    t.per = (int)((p.steps + S - 1) / S);
    S = (p.steps + t.per - 1) / t.per;
    t.S = (int)S;
    t.units = S > 1 ? (int)(tail * S) : 0;
    t.full = (int)(S > 1 ? tiles - tail : tiles);
    p.S = 1;
  }
  p.xp = 0;
  p.rs = p.kind != AwqPlan::kTiles ? 0 : align256((size_t)((M + 15) / 16) * p.steps * p.terms * 4096);
  p.partials = p.kind != AwqPlan::kTiles ? 0 : p.rs + align256((size_t)(M + 15) / 16 * 16 * 4);
  p.total = p.partials + (p.S > 1 ? align256((size_t)p.S * M * N * 4) : 0) + (size_t)p.t.units * 16 * p.t.mt * kGemmCols * 4;
  return p;
}

template <int XT, int TERMS>
void pack_rows(int M, int K, int steps, const void* x, uint8_t* xp, float* rs, hipStream_t st) {
  const int grid = ((M + 15) / 16 + 7) / 8 * 8 * 16;
  hipLaunchKernelGGL((awq_pack_kernel<XT, TERMS>), dim3(grid), dim3(256), 0, st, M, K, steps, x, xp, rs);
}

template <int ML, int XS, int MR>
hipError_t run_rows(const AwqPlan& p, int M, int N, int K, const void* x, const uint8_t* bank, const AwqLayout& L, float* y,
                    float* partials, hipStream_t st) {
  if (!raise_lds_limit<awq_rows_kernel<ML, XS, MR>>()) return hipErrorInvalidValue;
  const int sums = p.waves * M * 20 * 4, held = 16 * (K / 32) * ML + 32 + p.waves * MR * p.terms * 1024;
  hipLaunchKernelGGL((awq_rows_kernel<ML, XS, MR>), dim3((N + 15) / 16, p.S), dim3(64 * p.waves), std::max(sums, held), st, M, N, K,
                     RowsPlan{p.units, p.per, p.waves}, x, bank, L, y, partials);
  return hipGetLastError();
}
template <int ML, int XS, int CT>
hipError_t run_shared(const AwqPlan& p, int M, int N, int K, const void* x, const uint8_t* bank, const AwqLayout& L, float* y,
                      float* partials, hipStream_t st) {
  if (!raise_lds_limit<awq_shared_kernel<ML, XS, CT>>()) return hipErrorInvalidValue;
  const int sb = shared_blocks(CT * p.terms), lds = 16 * CT * p.terms * (sb * 1024 + 16) + kSharedWaves * 16 * sb * 16 * ML + 16 * CT * 4;
  hipLaunchKernelGGL((awq_shared_kernel<ML, XS, CT>), dim3((N + 16 * kSharedWaves - 1) / (16 * kSharedWaves), p.S), dim3(64 * kSharedWaves),
                     lds, st, M, N, K, p.units, p.per, x, bank, L, y, partials);
  return hipGetLastError();
}
template <int ML, int TERMS, int MT>
hipError_t run_gemm(const AwqPlan& p, int M, int N, const void* xp, const float* rs, const uint8_t* bank, const AwqLayout& L,
                    float* y, float* partials, hipStream_t st) {
  if (!raise_lds_limit<awq_gemm_kernel<ML, TERMS, MT>>()) return hipErrorInvalidValue;
  const TilePlan& t = p.t;
  hipLaunchKernelGGL((awq_gemm_kernel<ML, TERMS, MT>), dim3((t.full + 7) / 8 * 8 + (t.units + 7) / 8 * 8), dim3(256),
                     2 * MT * TERMS * 4096, st, M, N, t, static_cast<const uint8_t*>(xp), rs, bank, L, y, partials);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || t.units == 0) return e;
  hipLaunchKernelGGL(awq_tiles_join_kernel, dim3((unsigned)(t.units / t.S) * 16 * MT), dim3(256), 0, st, M, N, t, partials, y);
  return hipGetLastError();
}
// x: its terms and rs their scales (kTiles), else x itself.
template <int ML, int XT>
hipError_t run_plan(const AwqPlan& p, int M, int N, int K, const void* x, const float* rs, const uint8_t* bank, const AwqLayout& L, float* y,
                    float* partials, hipStream_t st) {
  constexpr int T = XT == X_F32 ? 2 : 1;
  switch (p.kind) {
    case AwqPlan::kOwn:
      if (M == 1) return run_rows<ML, XT, 1>(p, M, N, K, x, bank, L, y, partials, st);
      return run_rows<ML, XT, 2>(p, M, N, K, x, bank, L, y, partials, st);
    case AwqPlan::kShared:
      return p.ct == 1 ? run_shared<ML, XT, 1>(p, M, N, K, x, bank, L, y, partials, st)
                       : run_shared<ML, XT, 2>(p, M, N, K, x, bank, L, y, partials, st);
    default: break;
  }
  if constexpr (T == 1)
    if (p.t.mt == 8) return run_gemm<ML, T, 8>(p, M, N, x, rs, bank, L, y, partials, st);
  return run_gemm<ML, T, 4>(p, M, N, x, rs, bank, L, y, partials, st);
}
template <int XT>
hipError_t linear(const AwqPlan& p, int M, int N, int K, const void* x, const uint8_t* bank, int meta_layout, uint8_t* ws, float* y,
                  hipStream_t st) {
  const AwqLayout L = awq_layout(N, K, meta_layout);
  uint8_t* xp = ws + p.xp;
  float* rs = reinterpret_cast<float*>(ws + p.rs);
  float* partials = p.S > 1 || p.t.units > 0 ? reinterpret_cast<float*>(ws + p.partials) : nullptr;
  if (p.kind == AwqPlan::kTiles) {
    pack_rows<XT, XT == X_F32 ? 2 : 1>(M, K, p.steps, x, xp, rs, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    x = xp;
  }
  const hipError_t e = meta_layout == 3 ? run_plan<3, XT>(p, M, N, K, x, rs, bank, L, y, partials, st)
                                        : run_plan<4, XT>(p, M, N, K, x, rs, bank, L, y, partials, st);
  if (e != hipSuccess || p.S == 1) return e;
  hipLaunchKernelGGL(awq_join_kernel, dim3((N + 255) / 256, M), dim3(256), 0, st, M, N, p.S, partials, y);
  return hipGetLastError();
}

}  // namespace

size_t awq_linear_scratch_bytes(int M, int N, int K, XType xt) { return M == 0 ? 0 : awq_plan(M, N, K, xt).total; }

hipError_t launch_awq_linear(int M, int N, int K, const void* x, XType xt, const uint8_t* bank, int meta_layout, void* ws, float* y,
                             hipStream_t st) {
  const AwqPlan p = awq_plan(M, N, K, xt);
  uint8_t* base = static_cast<uint8_t*>(ws);
  if (xt == X_F32) return linear<X_F32>(p, M, N, K, x, bank, meta_layout, base, y, st);
  if (xt == X_BF16) return linear<X_BF16>(p, M, N, K, x, bank, meta_layout, base, y, st);
  return linear<X_F16>(p, M, N, K, x, bank, meta_layout, base, y, st);
}

}  // namespace wq
