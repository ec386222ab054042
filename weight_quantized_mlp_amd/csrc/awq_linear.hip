// Linear with AWQ int4 group-32 weights (gfx950): awq_linear_run in include/wqmlp_blocks.h,
//   y[m,n] = sum_k x[m,k] dq[n,k],  dq = RN_f16(q scale + bias) exactly as the routed step decodes it.
//
// The weights are decoded in registers, straight from the packed bytes, into matrix-core operands (awq_common.h); x is
// turned into float16 terms once (awq_pack_kernel), in the order the matrix cores read it.
//   Up to kSkinnyRows rows (awq_skinny_kernel): the weights' bytes bound it.  A workgroup's 8 waves split the
//     contraction of the same weight rows and add up through LDS, so a few rows of weights still fill a CU; x comes
//     from L2 as whole fragments.
//   More rows (awq_gemm_kernel): the matrix cores bound it.  4 waves with 64 weight rows each share the tile of x through
//     LDS (global->LDS copies, two stages); every wave decodes only its own weights, once per tile row.
// Either splits the contraction over workgroups when there are few tiles; awq_join_kernel adds the parts in order.
#include <algorithm>

#include "awq_common.h"
#include "dev_common.h"
#include "launch.h"

namespace wq {

namespace {

constexpr int kSkinnyRows = 32;

// ---- x -> float16 terms in fragment order ------------------------------------------------------------------------
// xp[m / 16][step][term][i][lane][8]: lane = 16 * quarter + m % 16 holds octet i of group 4 step + quarter of row m.
// Zeros past K (up to a whole step) and past M (up to a whole 16 rows).
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

// ---- few rows ----------------------------------------------------------------------------------------------------
// RT tiles of 16 weight rows, CT tiles of 16 rows of x; part blockIdx.y of the steps.
template <int ML, int TERMS, int RT, int CT>
__global__ void __launch_bounds__(512) awq_skinny_kernel(int M, int N, int steps, int per, const uint8_t* __restrict__ xp,
                                                         const float* __restrict__ rowscale, const uint8_t* __restrict__ bank,
                                                         AwqLayout L, float* __restrict__ y, float* __restrict__ partials) {
  constexpr int COLS = 16 * RT + 4;                          // floats of an LDS row: n, padded
  extern __shared__ __attribute__((aligned(16))) float part[];   // [8 waves][16 CT][COLS]
  const AwqDecode dc = awq_decode_consts();
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = (int)blockIdx.x * 16 * RT, q = lane >> 4;
  const int s0 = (int)blockIdx.y * per, s1 = min(s0 + per, steps), last = s1 - 1;
  const uint8_t* codes[RT];
  int64_t row[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    row[r] = min(n0 + 16 * r + (lane & 15), N - 1);
    codes[r] = bank + row[r] * (L.G * 16);
  }
  f32x4 acc[RT][CT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Step {
    AwqStep w[RT];
    f16x8 x[CT][TERMS][4];
  };
  auto load = [&](int s, Step& d) {
    const int sc = min(s, last);
#pragma unroll
    for (int r = 0; r < RT; ++r) d.w[r] = awq_load<ML>(codes[r], bank, L, row[r], 4 * sc + q);
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) d.x[c][t][i] = *reinterpret_cast<const f16x8*>(xp + frag_at(c, steps, sc, TERMS, t, i, lane));
  };
  auto multiply = [&](int s, const Step& d) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      f16x2 s2, b2;
      awq_meta<ML>(d.w[r], 4 * s + q < (int)L.G, s2, b2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f16x8 w = awq_frag(d.w[r].c[i], s2, b2, dc);
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int t = 0; t < TERMS; ++t) acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, d.x[c][t][i], acc[r][c], 0, 0, 0);
      }
    }
  };
  int s = s0 + wave;
  if (s < s1) {
    Step a, b;
    load(s, a);
    for (; s + 8 < s1; s += 16) {
      load(s + 8, b);
      multiply(s, a);
      load(s + 16, a);
      multiply(s + 8, b);
    }
    if (s < s1) multiply(s, a);
  }
  // the waves' sums, in order
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < CT; ++c)
      *reinterpret_cast<f32x4*>(part + (wave * 16 * CT + 16 * c + (lane & 15)) * COLS + 16 * r + 4 * q) = acc[r][c];
  __syncthreads();
  for (int i = tid; i < 16 * CT * 16 * RT; i += 512) {
    const int m = i / (16 * RT), j = i - m * 16 * RT, n = n0 + j;
    if (m >= M || n >= N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += part[(w * 16 * CT + m) * COLS + j];
    if (partials != nullptr) partials[((size_t)blockIdx.y * M + m) * N + n] = v;
    else y[(size_t)m * N + n] = v * rowscale[m];
  }
}

// ---- many rows ---------------------------------------------------------------------------------------------------
// Tile: 16 MT rows of x by 256 weight rows, 64 per wave.
constexpr int kGemmCols = 256;

template <int ML, int TERMS, int MT>
__global__ void __launch_bounds__(256, 2) awq_gemm_kernel(int M, int N, int steps, int per, int ntm, int tiles,
                                                          const uint8_t* __restrict__ xp, const float* __restrict__ rowscale,
                                                          const uint8_t* __restrict__ bank, AwqLayout L, float* __restrict__ y,
                                                          float* __restrict__ partials) {
  constexpr int NT = 4, UNITS = MT * TERMS, STAGE = UNITS * 4096;   // a unit: one term of 16 rows, 4 KB per step
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const AwqDecode dc = awq_decode_consts();
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4;
  // Workgroup b runs on XCD b % 8: each XCD gets a contiguous run of tiles, in bands of 8 tile rows, so that the tiles in
  // flight there share rows and weights in its L2.
  const int b = (int)blockIdx.x, chunk = (int)gridDim.x >> 3;
  const int id = (b & 7) * chunk + (b >> 3);
  if (id >= tiles) return;
  const int ntn = (N + kGemmCols - 1) / kGemmCols;
  const int band = id / (8 * ntn), in = id - band * 8 * ntn, height = min(8, ntm - 8 * band);
  const int tm = 8 * band + in % height, tn = in / height;
  const int n0 = tn * kGemmCols + 64 * wave, mt0 = tm * MT, mtiles = (M + 15) >> 4;
  const int s0 = (int)blockIdx.y * per, s1 = min(s0 + per, steps), last = s1 - 1;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  const uint8_t* codes[NT];
  int64_t row[NT];
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    row[r] = min(n0 + 16 * r + (lane & 15), N - 1);
    codes[r] = bank + row[r] * (L.G * 16);
  }
  // unit u = wave + 4 j: term u % TERMS of 16-row tile u / TERMS (past the end: the last one again, not stored)
  auto copy_x = [&](int step, int stage) {
#pragma unroll
    for (int j = 0; j < UNITS / 4; ++j) {
      const int u = wave + 4 * j, mt = min(mt0 + u / TERMS, mtiles - 1);
      const uint8_t* src = xp + frag_at(mt, steps, step, TERMS, u % TERMS, 0, 0);
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
  AwqStep cur[NT], nxt[NT];
  auto load_w = [&](int step, AwqStep* d) {
#pragma unroll
    for (int r = 0; r < NT; ++r) d[r] = awq_load<ML>(codes[r], bank, L, row[r], 4 * step + q);
  };
  copy_x(s0, 0);
  load_w(s0, cur);
  wait_vmem<0>();
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    const int st = (s - s0) & 1, next = min(s + 1, last);
    load_w(next, nxt);
    if (s < last) copy_x(next, st ^ 1);
    f16x2 s2[NT], b2[NT];
#pragma unroll
    for (int r = 0; r < NT; ++r) awq_meta<ML>(cur[r], 4 * s + q < (int)L.G, s2[r], b2[r]);
    const uint8_t* xs = lds + st * STAGE + lane * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f16x8 w[NT];
#pragma unroll
      for (int r = 0; r < NT; ++r) w[r] = awq_frag(cur[r].c[i], s2[r], b2[r], dc);
#pragma unroll
      for (int c = 0; c < MT; ++c)
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          const f16x8 xf = *reinterpret_cast<const f16x8*>(xs + (c * TERMS + t) * 4096 + i * 1024);
#pragma unroll
          for (int r = 0; r < NT; ++r) acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[r], xf, acc[r][c], 0, 0, 0);
        }
    }
#pragma unroll
    for (int r = 0; r < NT; ++r) cur[r] = nxt[r];
    wait_vmem<0>();            // the next step's copies landed
    wait_lds();
    __syncthreads();
  }
  float* out = partials != nullptr ? partials + (size_t)blockIdx.y * M * N : y;
#pragma unroll
  for (int c = 0; c < MT; ++c) {
    const int m = 16 * (mt0 + c) + (lane & 15);
    if (m >= M) continue;
    const float rs = partials != nullptr ? 1.f : rowscale[m];
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const int n = n0 + 16 * r + 4 * q;
      const f32x4 v = acc[r][c];
      float* o = out + (size_t)m * N + n;
      if (n + 3 < N && (N & 3) == 0) {
        *reinterpret_cast<f32x4*>(o) = f32x4{v[0] * rs, v[1] * rs, v[2] * rs, v[3] * rs};
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < N) o[j] = v[j] * rs;
      }
    }
  }
}

// y = row scale times the sum of the S parts, in order.
__global__ void __launch_bounds__(256) awq_join_kernel(int M, int N, int S, const float* __restrict__ partials,
                                                       const float* __restrict__ rowscale, float* __restrict__ y) {
  const int n = (int)blockIdx.x * 256 + (int)threadIdx.x, m = (int)blockIdx.y;
  if (n >= N) return;
  const size_t at = (size_t)m * N + n, part = (size_t)M * N;
  float v = partials[at];
  for (int s = 1; s < S; ++s) v += partials[s * part + at];
  y[at] = v * rowscale[m];
}

// ---- plan --------------------------------------------------------------------------------------------------------
struct AwqPlan {
  bool skinny;
  int terms, steps, S, per;
  int rt, ct;                  // skinny: row tiles, column tiles
  int mt, ntm, tiles;          // gemm
  size_t xp, rs, partials, total;
};
inline AwqPlan awq_plan(int M, int N, int K, XType xt) {
  AwqPlan p{};
  p.terms = awq_terms(xt);
  p.steps = (K + kStepK - 1) / kStepK;
  p.skinny = M <= kSkinnyRows;
  int64_t wgs;
  int want, least;             // workgroups that fill the chip; least steps of a part
  if (p.skinny) {
    p.ct = M <= 16 ? 1 : 2;
    p.rt = N >= 16 * 1024 ? 4 : (N >= 4096 ? 2 : 1);
    wgs = (N + 16 * p.rt - 1) / (16 * p.rt);
    want = 512, least = 32;    // four steps for each of the 8 waves
  } else {
    p.mt = p.terms == 2 || M <= 64 ? 4 : 8;
    p.ntm = (M + 16 * p.mt - 1) / (16 * p.mt);
    p.tiles = p.ntm * ((N + kGemmCols - 1) / kGemmCols);
    wgs = p.tiles;
    want = 512, least = 4;
  }
  int64_t S = std::max<int64_t>(1, std::min<int64_t>(want / wgs, p.steps / least));
  S = std::min<int64_t>(S, std::max<int64_t>(1, ((int64_t)64 << 20) / ((int64_t)M * N * 4)));   // at most 64 MiB of parts
  p.per = (int)((p.steps + S - 1) / S);
  p.S = (p.steps + p.per - 1) / p.per;
  p.xp = 0;
  p.rs = align256((size_t)((M + 15) / 16) * p.steps * p.terms * 4096);
  p.partials = p.rs + align256((size_t)(M + 15) / 16 * 16 * 4);
  p.total = p.partials + (p.S > 1 ? align256((size_t)p.S * M * N * 4) : 0);
  return p;
}

template <int XT, int TERMS>
void pack_rows(int M, int K, int steps, const void* x, uint8_t* xp, float* rs, hipStream_t st) {
  const int grid = ((M + 15) / 16 + 7) / 8 * 8 * 16;
  hipLaunchKernelGGL((awq_pack_kernel<XT, TERMS>), dim3(grid), dim3(256), 0, st, M, K, steps, x, xp, rs);
}

template <int ML, int TERMS, int RT, int CT>
hipError_t run_skinny(const AwqPlan& p, int M, int N, const uint8_t* xp, const float* rs, const uint8_t* bank, const AwqLayout& L,
                      float* y, float* partials, hipStream_t st) {
  if (!raise_lds_limit<awq_skinny_kernel<ML, TERMS, RT, CT>>()) return hipErrorInvalidValue;
  const int lds = 8 * 16 * CT * (16 * RT + 4) * 4;
  hipLaunchKernelGGL((awq_skinny_kernel<ML, TERMS, RT, CT>), dim3((N + 16 * RT - 1) / (16 * RT), p.S), dim3(512), lds, st, M, N,
                     p.steps, p.per, xp, rs, bank, L, y, partials);
  return hipGetLastError();
}
template <int ML, int TERMS, int MT>
hipError_t run_gemm(const AwqPlan& p, int M, int N, const uint8_t* xp, const float* rs, const uint8_t* bank, const AwqLayout& L,
                    float* y, float* partials, hipStream_t st) {
  if (!raise_lds_limit<awq_gemm_kernel<ML, TERMS, MT>>()) return hipErrorInvalidValue;
  hipLaunchKernelGGL((awq_gemm_kernel<ML, TERMS, MT>), dim3((p.tiles + 7) / 8 * 8, p.S), dim3(256), 2 * MT * TERMS * 4096, st, M, N,
                     p.steps, p.per, p.ntm, p.tiles, xp, rs, bank, L, y, partials);
  return hipGetLastError();
}
template <int ML, int TERMS, typename... A>
hipError_t run_plan(const AwqPlan& p, A... a) {
  if (!p.skinny) {
    if constexpr (TERMS == 1)
      if (p.mt == 8) return run_gemm<ML, TERMS, 8>(p, a...);
    return run_gemm<ML, TERMS, 4>(p, a...);
  }
  if (p.ct == 1) {
    if (p.rt == 4) return run_skinny<ML, TERMS, 4, 1>(p, a...);
    if (p.rt == 2) return run_skinny<ML, TERMS, 2, 1>(p, a...);
    return run_skinny<ML, TERMS, 1, 1>(p, a...);
  }
  if (p.rt == 4) return run_skinny<ML, TERMS, 4, 2>(p, a...);
  if (p.rt == 2) return run_skinny<ML, TERMS, 2, 2>(p, a...);
  return run_skinny<ML, TERMS, 1, 2>(p, a...);
}

}  // namespace

size_t awq_linear_scratch_bytes(int M, int N, int K, XType xt) { return M == 0 ? 0 : awq_plan(M, N, K, xt).total; }

hipError_t launch_awq_linear(int M, int N, int K, const void* x, XType xt, const uint8_t* bank, int meta_layout, void* ws, float* y,
                             hipStream_t st) {
  const AwqPlan p = awq_plan(M, N, K, xt);
  const AwqLayout L = awq_layout(N, K, meta_layout);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  uint8_t* xp = base + p.xp;
  float* rs = reinterpret_cast<float*>(base + p.rs);
  float* partials = p.S > 1 ? reinterpret_cast<float*>(base + p.partials) : nullptr;
  if (xt == X_F32) pack_rows<X_F32, 2>(M, K, p.steps, x, xp, rs, st);
  else if (xt == X_BF16) pack_rows<X_BF16, 1>(M, K, p.steps, x, xp, rs, st);
  else pack_rows<X_F16, 1>(M, K, p.steps, x, xp, rs, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (meta_layout == 3)
    e = p.terms == 2 ? run_plan<3, 2>(p, M, N, xp, rs, bank, L, y, partials, st) : run_plan<3, 1>(p, M, N, xp, rs, bank, L, y, partials, st);
  else
    e = p.terms == 2 ? run_plan<4, 2>(p, M, N, xp, rs, bank, L, y, partials, st) : run_plan<4, 1>(p, M, N, xp, rs, bank, L, y, partials, st);
  if (e != hipSuccess || partials == nullptr) return e;
  hipLaunchKernelGGL(awq_join_kernel, dim3((N + 255) / 256, M), dim3(256), 0, st, M, N, p.S, partials, rs, y);
  return hipGetLastError();
}

}  // namespace wq
