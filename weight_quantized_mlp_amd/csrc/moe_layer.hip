// Mixture-of-experts layer with AWQ int4 group-32 experts for a few tokens (gfx950): moe_awq_run in
// include/wqmlp_blocks.h.
//
//   router   logits[m,e] = RN_f32(sum_h x[m,h] router[e,h]) (summed in float64, so that which experts are chosen does not
//            depend on an order of additions), the topk largest, softmax                    route_* kernels
//   W13      act[r,i] = silu(g) u for every route r = (token, place), from the route's expert      moe_mm_kernel<true>
//   W2       y_r[o] = sum_i act[r,i] dq2[e][o,i]                                                  moe_mm_kernel<false>
//   sum      out[m,o] = sum over the token's routes, in order, of weight * y_r[o]                 moe_sum_kernel
//
// The experts' bytes bound it as soon as tokens spread over many experts, and every expert is read once for all of its
// tokens: a workgroup belongs to one expert (or to one route, the first that names its expert, when there are fewer routes
// than experts) and some of its rows, gathers the expert's routes from the list of ids, and multiplies its weights, decoded
// in registers (awq_common.h), with up to 16 of them at a time on the matrix cores.  Its 8 waves split the rows and the
// contraction.  act travels in float32 and enters W2 as two float16 terms, like float32 x, so nothing is rounded to 16 bits
// on the way.
#include <algorithm>

#include "awq_common.h"
#include "dev_common.h"
#include "launch.h"

namespace wq {

namespace {

// ---- router ------------------------------------------------------------------------------------------------------
// A wave per expert, kRouteTokens tokens at a time: 8 elements per lane and turn, products and sums in float64 (a product of
// two float32 is exact there).
constexpr int kRouteTokens = 4;

template <int XT, int WT>
__global__ void __launch_bounds__(256) route_logits_kernel(int M, int E, int H, const void* __restrict__ x,
                                                           const void* __restrict__ router, float* __restrict__ logits) {
  const int lane = (int)threadIdx.x & 63, e = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6), m0 = (int)blockIdx.y * kRouteTokens;
  if (e >= E) return;
  double acc[kRouteTokens] = {};
  for (int o = lane; o < H / 8; o += 64) {
    float w[8];
    load_octet<WT>(router, (size_t)e * H + 8 * (size_t)o, w);
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t) {
      float v[8];
      load_octet<XT>(x, (size_t)min(m0 + t, M - 1) * H + 8 * (size_t)o, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[t] = fma((double)v[j], (double)w[j], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kRouteTokens; ++t) {
    for (int off = 32; off >= 1; off >>= 1) acc[t] += __shfl_xor(acc[t], off, 64);
    if (lane == 0 && m0 + t < M) logits[(size_t)(m0 + t) * E + e] = (float)acc[t];
  }
}

// Order of selection as one number, larger first: the logit (NaN below everything, -0 as 0), then the lower index.
__device__ __forceinline__ uint64_t route_rank(float logit, int e) {
  const uint32_t b = __float_as_uint(logit + 0.f);
  const uint32_t key = logit == logit ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
  return ((uint64_t)key << 32) | (uint32_t)(0x7FFFFFFF - e);
}
// One wave: the topk largest of the token's E logits, each found as the largest one below the last.  Lane k gets the k-th
// (topk <= 16); the weights are the softmax of the chosen (renorm) or of all.
__device__ __forceinline__ void route_token(int E, int topk, bool renorm, const float* __restrict__ logits, int lane, int& id, float& weight) {
  uint64_t last = ~0ull;
  float first = 0.f, sum = 0.f, mine = 0.f;
  id = 0;
  for (int k = 0; k < topk; ++k) {
    uint64_t best = 0;
    for (int e = lane; e < E; e += 64) {
      const uint64_t r = route_rank(logits[e], e);
      if (r < last && r > best) best = r;
    }
    for (int off = 32; off >= 1; off >>= 1) {
      const uint64_t o = __shfl_xor((unsigned long long)best, off, 64);
      best = o > best ? o : best;
    }
    last = best;
    const int e = 0x7FFFFFFF - (int)(uint32_t)best;
    const float l = logits[e];
    if (k == 0) first = l;
    const float p = expf(l - first);
    sum += p;
    if (lane == k) {
      id = e;
      mine = p;
    }
  }
  if (!renorm) {
    sum = 0.f;
    for (int e = lane; e < E; e += 64) sum += expf(logits[e] - first);
    sum = group_sum<64>(sum);
  }
  weight = mine / sum;
}
__global__ void __launch_bounds__(256) route_topk_kernel(int M, int E, int topk, int renorm, const float* __restrict__ logits,
                                                         int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = (int)threadIdx.x & 63, m = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6);
  if (m >= M) return;
  int id;
  float w;
  route_token(E, topk, renorm != 0, logits + (size_t)m * E, lane, id, w);
  if (lane < topk) {
    ids[(size_t)m * topk + lane] = id;
    weights[(size_t)m * topk + lane] = w;
  }
}

// ---- the experts' products ---------------------------------------------------------------------------------------
constexpr int kMaxRoutes = 256 * 16;
constexpr int kPartRow = 20;                   // floats of a row of partial sums: 16, padded
constexpr int kColBytes = 16;                  // padding of a staged column
constexpr int kStageBytes = 16 * 2 * (8 * 256 + kColBytes);   // activations of one pass: 16 columns of two terms, a step for each
                                                              // of 8 waves; two workgroups share a CU
constexpr int kHeadBytes = kMaxRoutes * 2 + 16 * 4 + kMaxRoutes / 64 * 8;
constexpr int kMoeLds = kHeadBytes + kStageBytes;

struct MoeShape {
  int E, routes, topk;
  int K, rows;                 // contraction; rows of weights per expert (of gate, for W13)
  int wk;                      // waves that split the contraction (1, 2, 4 or 8); 8 / wk groups of rows per workgroup
  int by_route;                // blockIdx.y is a route, else an expert
};

// GU (W13): a wave's two row tiles are 16 gate rows and the same 16 up rows, src = x (row = token), dst = act [route][rows].
// Else (W2): 32 rows, src = act (row = route), dst = y [route][rows].
template <bool GU, int XT, int ML>
__global__ void __launch_bounds__(512) moe_mm_kernel(MoeShape sh, const void* __restrict__ src, const int32_t* __restrict__ ids,
                                                     const uint8_t* __restrict__ bank, AwqLayout L, float* __restrict__ dst) {
  constexpr int TERMS = XT == X_F32 ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint16_t* list = reinterpret_cast<uint16_t*>(lds);                              // the expert's routes, ascending
  float* scales = reinterpret_cast<float*>(lds + kMaxRoutes * 2);                 // of the pass's columns
  uint64_t* masks = reinterpret_cast<uint64_t*>(lds + kMaxRoutes * 2 + 16 * 4);   // of each 64 ids: those that name the expert
  uint8_t* stage = lds + kHeadBytes;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, item = (int)blockIdx.y;
  const int e = sh.by_route ? ids[item] : item;
  if (e < 0 || e >= sh.E) return;

  // The list: 64 ids per wave and turn, each match's place from the matches before it.
  const int blocks = (sh.routes + 63) >> 6;
  for (int b = wave; b < blocks; b += 8) {
    const int r = 64 * b + lane;
    const uint64_t mask = __ballot(r < sh.routes && ids[r] == e);
    if (lane == 0) masks[b] = mask;
  }
  __syncthreads();
  int nc = 0;
  for (int b = 0; b < blocks; ++b) {
    const uint64_t mask = masks[b];
    if (b % 8 == wave && (mask >> lane & 1)) list[nc + __popcll(mask & ((1ull << lane) - 1))] = (uint16_t)(64 * b + lane);
    nc += __popcll(mask);
  }
  __syncthreads();
  if (nc == 0 || (sh.by_route && (int)list[0] != item)) return;    // nobody's expert, or another route's workgroup has it

  const int wk = wave % sh.wk, group = (int)blockIdx.x * (8 / sh.wk) + wave / sh.wk, per = GU ? 16 : 32;
  const int groups = sh.rows / per, gc = min(group, groups - 1);
  const uint8_t* expert = bank + (size_t)e * L.expert_bytes;
  const uint8_t* codes[2];
  int64_t row[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    row[t] = gc * per + (lane & 15) + t * (GU ? sh.rows : 16);
    codes[t] = expert + row[t] * (L.G * 16);
  }
  const int steps = (sh.K + kStepK - 1) / kStepK, real = sh.K / 8;

  for (int c0 = 0; c0 < nc; c0 += 16) {
    const int cols = min(16, nc - c0);
    auto src_row = [&](int c) {
      const int r = list[c0 + c];
      return (size_t)(GU ? r / sh.topk : r) * sh.K;
    };
    __syncthreads();                                                // the last pass's readers of scales are done
    for (int c = wave; c < cols; c += 8) {                          // column c's power of two
      float amax = 0.f;
      if constexpr (XT != X_F16)
        for (int o = lane; o < real; o += 64) {
          float v[8];
          load_octet<XT>(src, src_row(c) + 8 * (size_t)o, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(v[j]));
        }
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
      if (lane == 0) scales[c] = XT == X_F16 ? 1.f : ldexpf(1.f, f16_row_exp(amax));
    }
    f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    // steps staged at a time: a multiple of wk, so that which wave takes which step, and with it the order of every sum, does
    // not depend on how many columns there are
    const int room = (kStageBytes / (cols * TERMS) - kColBytes) / (kStepK * 2), chunk = room >= steps ? steps : room / sh.wk * sh.wk;
    const int stride = chunk * kStepK * 2 + kColBytes;              // of one term of one column
    for (int k0 = 0; k0 < steps; k0 += chunk) {
      const int ks = min(chunk, steps - k0), end = k0 + ks;
      int s = k0 + wk;
      AwqStep a[2], b[2];
      auto load = [&](int step, AwqStep* d) {
        const int sc = min(step, steps - 1);
        d[0] = awq_load<ML>(codes[0], expert, L, row[0], 4 * sc + q);
        d[1] = awq_load<ML>(codes[1], expert, L, row[1], 4 * sc + q);
      };
      load(s, a);
      __syncthreads();                                              // scales written; the last chunk's readers done
      for (int i = tid; i < cols * ks * 16; i += 512) {
        const int c = i / (ks * 16), o = i - c * ks * 16, at = k0 * 16 + o;
        u32x4 w[TERMS];
        if (at < real) {
          float v[8];
          load_octet<XT>(src, src_row(c) + 8 * (size_t)at, v);
          int ex = 0;
          if constexpr (XT != X_F16) ex = (int)((__float_as_uint(scales[c]) >> 23) & 255) - 127;
          octet_terms<TERMS>(v, ex, w);
        } else {
#pragma unroll
          for (int t = 0; t < TERMS; ++t) w[t] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int t = 0; t < TERMS; ++t) *reinterpret_cast<u32x4*>(stage + (c * TERMS + t) * stride + o * 16) = w[t];
      }
      __syncthreads();
      const uint8_t* xs = stage + min(lane & 15, cols - 1) * TERMS * stride + q * 64;
      auto multiply = [&](int step, const AwqStep* d) {
        f16x2 s2[2], b2[2];
        const bool live = 4 * step + q < (int)L.G;
        awq_meta<ML>(d[0], live, s2[0], b2[0]);
        awq_meta<ML>(d[1], live, s2[1], b2[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f16x8 w0 = awq_frag(d[0].c[i], s2[0], b2[0]), w1 = awq_frag(d[1].c[i], s2[1], b2[1]);
#pragma unroll
          for (int t = 0; t < TERMS; ++t) {
            const f16x8 xf = *reinterpret_cast<const f16x8*>(xs + t * stride + (step - k0) * 256 + i * 16);
            acc[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0, xf, acc[0], 0, 0, 0);
            acc[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1, xf, acc[1], 0, 0, 0);
          }
        }
      };
      for (; s + sh.wk < end; s += 2 * sh.wk) {
        load(s + sh.wk, b);
        multiply(s, a);
        load(s + 2 * sh.wk, a);
        multiply(s + sh.wk, b);
      }
      if (s < end) multiply(s, a);
    }
    __syncthreads();                                                // the stage becomes the waves' partial sums
    float* part = reinterpret_cast<float*>(stage);                  // [wave][tile][column][16 rows]
#pragma unroll
    for (int t = 0; t < 2; ++t)
      *reinterpret_cast<f32x4*>(part + ((wave * 2 + t) * 16 + (lane & 15)) * kPartRow + 4 * q) = acc[t];
    __syncthreads();
    const int wr = 8 / sh.wk;
    for (int i = tid; i < wr * cols * per; i += 512) {
      const int n = i % per, c = (i / per) % cols, g = i / (per * cols), out = ((int)blockIdx.x * wr + g) * per + n;
      if (out >= sh.rows) continue;
      const int tile = GU ? 0 : n >> 4;
      float v = 0.f, u = 0.f;
      for (int w = 0; w < sh.wk; ++w) {
        const float* p = part + (((g * sh.wk + w) * 2 + tile) * 16 + c) * kPartRow + (n & 15);
        v += p[0];
        if constexpr (GU) u += p[16 * kPartRow];
      }
      v *= scales[c];
      if constexpr (GU) v = silu_f32(v) * (u * scales[c]);
      dst[(size_t)list[c0 + c] * sh.rows + out] = v;
    }
  }
}

// ---- sum over a token's routes -----------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) moe_sum_kernel(int E, int topk, int H, const int32_t* __restrict__ ids,
                                                      const float* __restrict__ weights, const float* __restrict__ y, void* __restrict__ out,
                                                      int ot) {
  const int m = (int)blockIdx.y, o = 4 * ((int)blockIdx.x * 256 + (int)threadIdx.x);
  if (o >= H) return;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < topk; ++k) {
    const int r = m * topk + k, e = ids[r];
    if (e < 0 || e >= E) continue;
    const float w = weights[r];
    const f32x4 p = *reinterpret_cast<const f32x4*>(y + (size_t)r * H + o);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = fmaf(w, p[j], v[j]);
  }
  const size_t at = (size_t)m * H + o;
  if (ot == X_F32) {
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out) + at) = v;
  } else {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = ot == X_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)v[j]) : __builtin_bit_cast(uint16_t, (_Float16)v[j]);
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(out) + at) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
  }
}

struct MoeWs {
  size_t logits, act, y, total;
};
inline MoeWs moe_ws(int M, int E, int topk, int H, int I) {
  MoeWs w;
  w.logits = 0;
  w.act = align256((size_t)M * E * 4);
  w.y = w.act + align256((size_t)M * topk * I * 4);
  w.total = w.y + align256((size_t)M * topk * H * 4);
  return w;
}

// Waves over the contraction: as many as leave each of them two steps or more.
inline int waves_over_k(int K) {
  const int steps = (K + kStepK - 1) / kStepK;
  return steps >= 16 ? 8 : (steps >= 8 ? 4 : (steps >= 4 ? 2 : 1));
}

template <bool GU, int XT, int ML>
hipError_t run_mm(const MoeShape& sh, int items, const void* src, const int32_t* ids, const uint8_t* bank, const AwqLayout& L, float* dst,
                  hipStream_t st) {
  if (!raise_lds_limit<moe_mm_kernel<GU, XT, ML>>()) return hipErrorInvalidValue;
  const int groups = sh.rows / (GU ? 16 : 32), wr = 8 / sh.wk;
  hipLaunchKernelGGL((moe_mm_kernel<GU, XT, ML>), dim3((groups + wr - 1) / wr, items), dim3(512), kMoeLds, st, sh, src, ids, bank, L,
                     dst);
  return hipGetLastError();
}
template <int ML>
hipError_t run_experts(int M, int E, int topk, int H, int I, const void* x, XType xt, const int32_t* ids, const uint8_t* w13,
                       const uint8_t* w2, float* act, float* y, hipStream_t st) {
  const int routes = M * topk, by_route = routes < E, items = std::min(routes, E);
  const MoeShape s13{E, routes, topk, H, I, waves_over_k(H), by_route}, s2{E, routes, topk, I, H, waves_over_k(I), by_route};
  const AwqLayout L13 = awq_layout(2 * (int64_t)I, H, ML), L2 = awq_layout(H, I, ML);
  hipError_t e = xt == X_F32    ? run_mm<true, X_F32, ML>(s13, items, x, ids, w13, L13, act, st)
                 : xt == X_BF16 ? run_mm<true, X_BF16, ML>(s13, items, x, ids, w13, L13, act, st)
                                : run_mm<true, X_F16, ML>(s13, items, x, ids, w13, L13, act, st);
  if (e != hipSuccess) return e;
  return run_mm<false, X_F32, ML>(s2, items, act, ids, w2, L2, y, st);
}
template <int XT>
void run_logits(int M, int E, int H, const void* x, const void* router, XType rt, float* logits, hipStream_t st) {
  const dim3 grid((E + 3) / 4, (M + kRouteTokens - 1) / kRouteTokens);
  if (rt == X_F32) hipLaunchKernelGGL((route_logits_kernel<XT, X_F32>), grid, dim3(256), 0, st, M, E, H, x, router, logits);
  else if (rt == X_BF16) hipLaunchKernelGGL((route_logits_kernel<XT, X_BF16>), grid, dim3(256), 0, st, M, E, H, x, router, logits);
  else hipLaunchKernelGGL((route_logits_kernel<XT, X_F16>), grid, dim3(256), 0, st, M, E, H, x, router, logits);
}

}  // namespace

size_t moe_awq_scratch_bytes(int M, int E, int topk, int H, int I) { return M == 0 ? 0 : moe_ws(M, E, topk, H, I).total; }

hipError_t launch_moe_awq(int M, int E, int topk, int H, int I, const void* x, XType xt, const void* router, XType rt, bool renorm,
                          int32_t* ids, float* weights, const uint8_t* w13, const uint8_t* w2, int meta_layout, void* ws, void* out,
                          XType ot, hipStream_t st) {
  const MoeWs W = moe_ws(M, E, topk, H, I);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  float* logits = reinterpret_cast<float*>(base + W.logits);
  float* act = reinterpret_cast<float*>(base + W.act);
  float* y = reinterpret_cast<float*>(base + W.y);
  hipError_t e;
  if (router != nullptr) {
    if (xt == X_F32) run_logits<X_F32>(M, E, H, x, router, rt, logits, st);
    else if (xt == X_BF16) run_logits<X_BF16>(M, E, H, x, router, rt, logits, st);
    else run_logits<X_F16>(M, E, H, x, router, rt, logits, st);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(route_topk_kernel, dim3((M + 3) / 4), dim3(256), 0, st, M, E, topk, renorm ? 1 : 0, logits, ids, weights);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  e = meta_layout == 3 ? run_experts<3>(M, E, topk, H, I, x, xt, ids, w13, w2, act, y, st)
                       : run_experts<4>(M, E, topk, H, I, x, xt, ids, w13, w2, act, y, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_sum_kernel, dim3((H + 1023) / 1024, M), dim3(256), 0, st, E, topk, H, ids, weights, y, out, (int)ot);
  return hipGetLastError();
}

}  // namespace wq
