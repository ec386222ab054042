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
// in registers (awq_common.h), with up to 16 of them at a time on the matrix cores.  act travels in float32 and enters W2 as
// two float16 terms, like float32 x, so nothing is rounded to 16 bits on the way.
//
// Calls in a row, 512 experts of 160 on 2560, 10 per token: 1 token 25 us (logits 4.7, choice 4, W13 8.4, W2 5.7, sum 3: five
// launches, each near what a launch with its chain of loads takes), 37 tokens 96 us for 195 MB (10, 5, 43, 33, 5).  64 experts of 704
// on 1024, 130 float32 tokens, 6 each: 73 us (6, 4, 37, 24, 5).  In W13 of 37 tokens half of the CUs' issue slots go to the decode
// and what surrounds it, a quarter of the time some CUs have run out of work.
#include <algorithm>

#include "awq_common.h"
#include "dev_common.h"
#include "launch.h"

namespace wq {

namespace {

// ---- router ------------------------------------------------------------------------------------------------------
// A wave for TE experts and TT tokens: 8 elements per lane and turn, products and sums in float64 (a product of two float32 is exact
// there), every element converted once.  Which elements a lane sums in which order does not depend on TE and TT.  (On the float64 matrix
// cores, 16 x 16 tiles: as fast for 37 tokens, 10.3 us for 512 experts on 2560, but 10.3 in place of 4.4 for one.)
template <int XT, int WT, int TE, int TT>
__global__ void __launch_bounds__(256) route_logits_kernel(int M, int E, int H, const void* __restrict__ x,
                                                           const void* __restrict__ router, float* __restrict__ logits) {
  const int lane = (int)threadIdx.x & 63, e0 = ((int)blockIdx.x * 4 + ((int)threadIdx.x >> 6)) * TE, m0 = (int)blockIdx.y * TT;
  if (e0 >= E) return;
  constexpr int UP = TT == 1 ? 4 : 2;                           // turns on their way at once
  double acc[TE][TT] = {};
  const int octets = H / 8;
  for (int o0 = lane; o0 < octets; o0 += 64 * UP) {
    RawOctet<WT> w[UP][TE];
    RawOctet<XT> v[UP][TT];
#pragma unroll
    for (int k = 0; k < UP; ++k) {
      const size_t at = 8 * (size_t)min(o0 + 64 * k, octets - 1);
#pragma unroll
      for (int i = 0; i < TE; ++i) w[k][i] = load_raw<WT>(router, (size_t)min(e0 + i, E - 1) * H + at);
#pragma unroll
      for (int t = 0; t < TT; ++t) v[k][t] = load_raw<XT>(x, (size_t)min(m0 + t, M - 1) * H + at);
    }
#pragma unroll
    for (int k = 0; k < UP; ++k) {
      if (o0 + 64 * k >= octets) break;
      double wd[TE][8];
#pragma unroll
      for (int i = 0; i < TE; ++i) {
        float f[8];
        raw_values<WT>(w[k][i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) wd[i][j] = f[j];
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        float f[8];
        raw_values<XT>(v[k][t], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double xd = f[j];
#pragma unroll
          for (int i = 0; i < TE; ++i) acc[i][t] = fma(xd, wd[i][j], acc[i][t]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TE; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      for (int off = 32; off >= 1; off >>= 1) acc[i][t] += __shfl_xor(acc[i][t], off, 64);
      if (lane == 0 && m0 + t < M && e0 + i < E) logits[(size_t)(m0 + t) * E + e0 + i] = (float)acc[i][t];
    }
}

// Order of selection as a signed number, larger first: NaN below every value, -0 as 0.  kTaken is below all.
constexpr int kTaken = -0x7FFFFFFF - 1;
__device__ __forceinline__ int route_key(float logit) {
  const int b = __float_as_int(logit + 0.f);
  return logit == logit ? (b < 0 ? b ^ 0x7FFFFFFF : b) : kTaken + 1;
}
__device__ __forceinline__ float route_logit(int key) {
  return key == kTaken + 1 ? __int_as_float(0x7FC00000) : __int_as_float(key < 0 ? key ^ 0x7FFFFFFF : key);
}
template <int CTRL>
__device__ __forceinline__ int dpp_i32(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true); }
__device__ __forceinline__ int wave64_max_i32(int v) {
  v = max(v, dpp_i32<0xB1>(v));
  v = max(v, dpp_i32<0x4E>(v));
  v = max(v, dpp_i32<0x141>(v));
  v = max(v, dpp_i32<0x140>(v));
  return max(max(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
             max(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}
// One wave per token: lane holds the keys of experts lane, lane + 64, ... (VPL of them, or VPL = 0: any number, read again for every
// choice).  Each turn takes the largest key, of equal ones the lowest expert.  Lane k gets the k-th choice; the weights are the softmax of
// the chosen (renorm) or of all.
template <int VPL>
__global__ void __launch_bounds__(64) route_topk_kernel(int E, int topk, int renorm, const float* __restrict__ all, int32_t* __restrict__ ids,
                                                        float* __restrict__ weights) {
  const int lane = (int)threadIdx.x, m = (int)blockIdx.x;
  const float* logits = all + (size_t)m * E;
  int key[VPL > 0 ? VPL : 1];
  if constexpr (VPL > 0) {
    float l[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) l[j] = logits[min(lane + 64 * j, E - 1)];
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = lane + 64 * j < E ? route_key(l[j]) : kTaken;
  }
  int id = 0, last_key = 0x7FFFFFFF, last_e = -1;
  float first = 0.f, mine = 0.f;
  for (int k = 0; k < topk; ++k) {
    int best = kTaken, at = 0x7FFFFFFF;                       // the lane's largest key and its expert
    if constexpr (VPL > 0) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (key[j] > best) best = key[j], at = lane + 64 * j;
    } else {
      for (int e = lane; e < E; e += 64) {
        const int v = route_key(logits[e]);
        const bool left = v < last_key || (v == last_key && e > last_e);
        if (left && v > best) best = v, at = e;
      }
    }
    const int top = wave64_max_i32(best);
    const uint64_t who = __ballot(best == top);               // seldom more than one lane
    const int e = (who & (who - 1)) == 0 ? __builtin_amdgcn_readlane(at, __builtin_ctzll(who))
                                         : -wave64_max_i32(best == top ? -at : -0x7FFFFFFF);
    if constexpr (VPL > 0) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (e == lane + 64 * j) key[j] = kTaken;
    }
    last_key = top, last_e = e;
    if (k == 0) first = route_logit(top);
    if (lane == k) id = e, mine = route_logit(top);
  }
  mine = lane < topk ? expf(mine - first) : 0.f;
  float sum = 0.f;
  if (renorm == 0)
    for (int e = lane; e < E; e += 64) sum += expf(logits[e] - first);
  sum = wave64_sum(renorm == 0 ? sum : mine);
  if (lane < topk) {
    ids[(size_t)m * topk + lane] = id;
    weights[(size_t)m * topk + lane] = mine / sum;
  }
}

// ---- the experts' products ---------------------------------------------------------------------------------------
// A pair is two tiles of 16 weight rows: W13 16 gate rows and the same 16 up rows, W2 32 rows.  A workgroup has some pairs of one
// expert: it finds the expert's routes in the list of ids, copies its rows' scales and zeros (contiguous pieces of the bank) to LDS,
// turns up to `cols` of the routes' rows into float16 terms there, 512 k at a time with a power of two of their own, and multiplies.
//   Many routes: a wave takes whole pairs, block after block of 512 k, each step's codes replaced by the next block's as soon as
//     they are used, and nothing is exchanged between waves.
//   Few routes (SPLIT): the waves of a workgroup share one pair's blocks, so that a workgroup needs no more than one pair: 10 routes of
//     160 on 2560 are 100 workgroups of 5 waves in W13.
// Either way a column's blocks are added in order, each scaled by a power of two, which is exact: its bits depend neither on the way nor on
// how many columns there are.
constexpr int kPartRow = 20;                   // floats of a row of partial sums: 16, padded
constexpr int kBlockK = 512, kBlockSteps = 4;

struct MoeShape {
  int E, routes, topk;
  int K, rows;                 // contraction; rows of weights per expert (of gate, for W13)
  int pairs;                   // of a workgroup
  int waves, cols;
  int by_route;                // blockIdx.y is a route, else an expert
};
// LDS: metadata, then the terms [cols][blocks][TERMS][1 KB] and their powers of two [cols][blocks], SPLIT: the blocks' sums
// [block][tile][cols][kPartRow], then the list of routes.
struct MoeLds {
  int terms, scales, part, list, total;
};
__host__ __device__ inline MoeLds moe_lds(const MoeShape& s, int terms, int ml, bool split) {
  MoeLds l;
  const int blocks = (s.K + kBlockK - 1) / kBlockK;
  l.terms = 2 * 16 * s.pairs * (s.K / 32) * ml;
  l.scales = l.terms + s.cols * blocks * terms * 1024;
  l.part = (l.scales + s.cols * blocks * 4 + 15) / 16 * 16;
  l.list = l.part + (split ? blocks * 2 * s.cols * kPartRow * 4 : 0);
  l.total = (l.list + s.routes * 2 + 15) / 16 * 16;
  return l;
}

// GU (W13): src = x (row = token), dst = act [route][rows].  Else (W2): src = act (row = route), dst = y [route][rows].
template <bool GU, bool SPLIT, int XT, int ML>
__global__ void __launch_bounds__(1024) moe_mm_kernel(MoeShape sh, const void* __restrict__ src, const int32_t* __restrict__ ids,
                                                     const uint8_t* __restrict__ bank, AwqLayout L, float* __restrict__ dst) {
  constexpr int TERMS = XT == X_F32 ? 2 : 1, ZB = ML == 3 ? 1 : 2;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const MoeLds at = moe_lds(sh, TERMS, ML, SPLIT);
  float* scales = reinterpret_cast<float*>(lds + at.scales);
  uint16_t* list = reinterpret_cast<uint16_t*>(lds + at.list);                 // the expert's routes, ascending
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, item = (int)blockIdx.y, T = 64 * sh.waves;

  // The expert's routes, 8 x 64 ids at a time.  Every wave finds them for itself and writes the same list, so none waits for another.
  int e = item, nc = 0;
  for (int r0 = 0; r0 < sh.routes; r0 += 512) {
    int id[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) id[k] = ids[min(r0 + 64 * k + lane, sh.routes - 1)];
    if (r0 == 0 && sh.by_route) e = ids[item];
    e = __builtin_amdgcn_readfirstlane(e);
    if (e < 0 || e >= sh.E) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = r0 + 64 * k + lane;
      const uint64_t mask = __ballot(r < sh.routes && id[k] == e);
      if (nc == 0 && mask != 0 && sh.by_route && r0 + 64 * k + __builtin_ctzll(mask) != item) return;   // an earlier route's workgroup has it
      if (mask >> lane & 1) list[nc + __popcll(mask & ((1ull << lane) - 1))] = (uint16_t)r;
      nc += __popcll(mask);
    }
  }
  if (nc == 0) return;
  wave_lds_fence();

  const int per = GU ? 16 : 32, G = (int)L.G, steps = (sh.K + kStepK - 1) / kStepK, blocks = (steps + kBlockSteps - 1) / kBlockSteps;
  const int p0 = (int)blockIdx.x * sh.pairs, p1 = min(p0 + sh.pairs, sh.rows / per);
  const uint8_t* expert = bank + (size_t)e * L.expert_bytes;
  // Tile t of pair p: rows tile_row(p, t) .. + 15 of the matrix.  Tiles 0 of the pairs, then tiles 1, lie in LDS as they do in the bank.
  auto tile_row = [&](int p, int t) { return GU ? 16 * p + t * sh.rows : 32 * p + 16 * t; };
  u32x4 c[2][4];                                                               // [tile][step] of a block
  auto load_step = [&](int p, int b, int s) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* tile = expert + (size_t)tile_row(p, t) * (G * 16);
      c[t][s] = *reinterpret_cast<const u32x4*>(tile + (uint32_t)((lane & 15) * G * 16 + 16 * min(16 * b + 4 * s + q, G - 1)));
    }
  };
  auto load = [&](int p, int b) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (s < steps - kBlockSteps * b) load_step(p, b, s);
  };
  const int kw = SPLIT ? wave : 0;
  int p = SPLIT ? p0 : p0 + wave;
  // Terms of a pass's columns: unit u is block u % blocks of column u / blocks, a wave takes every waves-th unit, two at a time.
  const int octets = sh.K / 8;
  constexpr int XU = 2;
  RawOctet<XT> raw[XU];
  auto load_units = [&](int c0, int units, int u0) {
#pragma unroll
    for (int k = 0; k < XU; ++k) {
      const int u = min(u0 + k * sh.waves, units - 1), col = u / blocks, o = 64 * (u - col * blocks) + lane;
      const int r = __builtin_amdgcn_readfirstlane((int)list[c0 + col]);
      const uint8_t* xrow = static_cast<const uint8_t*>(src) + (size_t)(GU ? r / sh.topk : r) * sh.K * (XT == X_F32 ? 4 : 2);
      raw[k] = load_raw<XT>(xrow, (uint32_t)(8 * min(o, octets - 1)));
    }
  };
  auto put_units = [&](int units, int u0) {
#pragma unroll
    for (int k = 0; k < XU; ++k) {
      const int u = u0 + k * sh.waves;
      if (u >= units) break;
      u32x4 t[TERMS];
      const float scale = wave_terms<XT, TERMS>(raw[k], 64 * (u % blocks) + lane < octets, t);
      uint8_t* to = lds + at.terms + u * (TERMS * 1024) + lane * 16;
#pragma unroll
      for (int j = 0; j < TERMS; ++j) *reinterpret_cast<u32x4*>(to + j * 1024) = t[j];
      if (lane == 0) scales[u] = scale;
    }
  };
  auto stage = [&](int c0) {                                                   // (the first two units are on their way)
    const int units = min(sh.cols, nc - c0) * blocks;
    for (int u0 = wave; u0 < units; u0 += XU * sh.waves) {
      if (u0 != wave) load_units(c0, units, u0);
      put_units(units, u0);
    }
  };
  load_units(0, min(sh.cols, nc) * blocks, wave);
  // Metadata of 16 np rows per piece: [tile 0: scales, zeros][tile 1: scales, zeros] for W13, one run of 32 np rows for W2.
  const int np = p1 - p0, runs = GU ? 2 : 1, run_rows = (GU ? 16 : 32) * np, sp = run_rows * G * 2 / 16, zp = run_rows * G * ZB / 16;
  {
    constexpr int UP = 4;
    const int pieces = runs * (sp + zp);
    u32x4 v[UP];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int k = 0; k < UP; ++k) {
        const int i = min(i0 + k * T, pieces - 1);
        const bool second = i >= sp + zp;
        const int j = second ? i - (sp + zp) : i;
        const size_t row = (size_t)(second ? sh.rows + 16 * p0 : per * p0);
        const uint8_t* from = j < sp ? expert + L.scale_off + row * G * 2 + 16 * (size_t)j
                                     : expert + L.meta2_off + row * G * ZB + 16 * (size_t)(j - sp);
        v[k] = *reinterpret_cast<const u32x4*>(from);
      }
    };
    fetch(tid);
    if (p < p1 && kw < blocks) load(p, kw);
    for (int i0 = tid; i0 < pieces; i0 += UP * T) {
      if (i0 != tid) fetch(i0);
#pragma unroll
      for (int k = 0; k < UP; ++k)
        if (i0 + k * T < pieces) reinterpret_cast<u32x4*>(lds)[i0 + k * T] = v[k];
    }
  }
  f32x4 acc[2], sum[2];
  for (int c0 = 0; c0 < nc; c0 += sh.cols) {
    const int cols = min(sh.cols, nc - c0);
    stage(c0);
    __syncthreads();
    const int mycol = min(lane & 15, cols - 1);
    const int route = list[c0 + mycol];
    // Block b of a pair; then its registers hold block b2 of pair p2 (p2 < 0: none).
    auto multiply = [&](int pair, int b, int p2, int b2) {
      const int ns = min(kBlockSteps, steps - kBlockSteps * b), ns2 = p2 < 0 ? 0 : steps - kBlockSteps * b2;
      const uint8_t* xs = lds + at.terms + (mycol * blocks + b) * (TERMS * 1024) + q * 64;
      sum[0] = sum[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s < ns) {
          const int g = 16 * b + 4 * s + q, gc = min(g, G - 1);
          f16x2 s2[2], b2[2];
  #pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int run = GU ? t * (sp + zp) * 16 : 0, row = (GU ? 16 * (pair - p0) : 32 * (pair - p0) + 16 * t) + (lane & 15);
            AwqStep a;
            a.s = *reinterpret_cast<const uint16_t*>(lds + run + (row * G + gc) * 2);
            if constexpr (ML == 3) a.z = lds[run + sp * 16 + row * G + gc];
            else a.z = *reinterpret_cast<const uint16_t*>(lds + run + sp * 16 + (row * G + gc) * 2);
            awq_meta<ML>(a, g < G, s2[t], b2[t]);
          }
  #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f16x8 w0 = awq_frag(c[0][s][i], s2[0], b2[0]), w1 = awq_frag(c[1][s][i], s2[1], b2[1]);
  #pragma unroll
            for (int j = 0; j < TERMS; ++j) {
              const f16x8 xf = *reinterpret_cast<const f16x8*>(xs + j * 1024 + s * 256 + i * 16);
              sum[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0, xf, sum[0], 0, 0, 0);
              sum[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1, xf, sum[1], 0, 0, 0);
            }
          }
        }
        if (s < ns2) load_step(p2, b2, s);
      }
      const float rs = scales[mycol * blocks + b];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[t][j] *= rs;
    };
    if constexpr (SPLIT) {
      float* part = reinterpret_cast<float*>(lds + at.part);
      for (int b = kw; b < blocks; b += sh.waves) {
        multiply(p0, b, b + sh.waves < blocks ? p0 : -1, b + sh.waves);
        if ((lane & 15) < cols)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            *reinterpret_cast<f32x4*>(part + ((b * 2 + t) * sh.cols + (lane & 15)) * kPartRow + 4 * q) = sum[t];
      }
      __syncthreads();
      for (int i = tid; i < cols * per; i += T) {
        const int n = i % per, col = i / per, t = GU ? 0 : n >> 4;
        float v = 0.f, u = 0.f;
        for (int b = 0; b < blocks; ++b) {
          const float* f = part + ((b * 2 + t) * sh.cols + col) * kPartRow + (n & 15);
          v += f[0];
          if constexpr (GU) u += f[sh.cols * kPartRow];
        }
        if constexpr (GU) v = silu_f32(v) * u;
        dst[(size_t)list[c0 + col] * sh.rows + per * p0 + n] = v;
      }
      if (c0 + sh.cols < nc && kw < blocks) load(p0, kw);                      // the next pass starts over
    } else {
      for (int pair = p, b = 0; pair < p1;) {
        int b2 = b + 1, p2 = pair;
        if (b2 == blocks) b2 = 0, p2 += sh.waves;
        multiply(pair, b, p2 < p1 ? p2 : (c0 + sh.cols < nc ? p : -1), b2);    // (the next pass starts over)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[t][j] = b == 0 ? sum[t][j] : acc[t][j] + sum[t][j];
        if (b2 == 0 && (lane & 15) < cols) {
          float* o = dst + (size_t)route * sh.rows + per * pair + 4 * q;
          if constexpr (GU) {
            f32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = silu_f32(acc[0][j]) * acc[1][j];
            *reinterpret_cast<f32x4*>(o) = v;
          } else {
            *reinterpret_cast<f32x4*>(o) = acc[0];
            *reinterpret_cast<f32x4*>(o + 16) = acc[1];
          }
        }
        b = b2, pair = p2;
      }
    }
    if (c0 + sh.cols >= nc) return;
    load_units(c0 + sh.cols, min(sh.cols, nc - c0 - sh.cols) * blocks, wave);
    __syncthreads();                                                           // the terms have been read
  }
}

// ---- sum over a token's routes -----------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) moe_sum_kernel(int E, int topk, int H, const int32_t* __restrict__ ids,
                                                      const float* __restrict__ weights, const float* __restrict__ y, void* __restrict__ out,
                                                      int ot) {
  const int m = (int)blockIdx.y, o = 4 * ((int)blockIdx.x * 256 + (int)threadIdx.x);
  if (o >= H) return;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  constexpr int UP = 8;                          // routes on their way at once, valid or not (one after the other: 1 token 4.4 us,
                                                 // so 3.0)
  for (int k0 = 0; k0 < topk; k0 += UP) {
    int e[UP];
    float w[UP];
    f32x4 p[UP];
#pragma unroll
    for (int k = 0; k < UP; ++k) {
      const int r = m * topk + min(k0 + k, topk - 1);
      e[k] = ids[r];
      w[k] = weights[r];
      p[k] = *reinterpret_cast<const f32x4*>(y + (size_t)r * H + o);
    }
#pragma unroll
    for (int k = 0; k < UP; ++k) {
      if (k0 + k >= topk || e[k] < 0 || e[k] >= E) continue;                   // (such a route's y is not written)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = fmaf(w[k], p[k][j], v[j]);
    }
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

// Columns of a pass: two and a half times what an expert has on average, in at most 64 KB of terms.  Pairs of a workgroup, in at most 48 KB
// of metadata (or one pair): few experts are cut into 260 workgroups, whose up to 16 waves share the columns' terms; many, with a column or
// two each, into 1200, of which several fit a CU.  130 rows, 64 experts of 704 on 1024: 260 73 us, 530 80, 800 94; 37 rows, 512 experts of
// 160 on 2560: 400 121 us, 800 103, 1200 97, 1600 109.  Where it changes: items are the experts or, if fewer, the routes; at 64, 128, 160
// and 256 of them (260 workgroups of up to 16 waves against 1200 of up to 8) bfloat16 experts of 160 on 2560 with a row each take 38 and 46 us,
// 45 and 54, 70 and 58, 86 and 73, of 512 on 2048 with two rows each 47 and 50, 77 and 82, 109 and 105, 138 and 132, float32 ones of 704 on
// 1024 with six rows each 48 and 67, 88 and 111, 120 and 123, 163 and 178 (these would keep the 260).
// The blocks are split over waves where whole pairs would leave the chip with less than two waves per CU.
struct MoePlan {
  MoeShape s;
  bool split;
};
inline MoePlan moe_plan(int E, int routes, int topk, int K, int rows, bool gu, int terms, int ml) {
  const int blocks = (K + kBlockK - 1) / kBlockK, all = rows / (gu ? 16 : 32), items = std::min(routes, E);
  MoePlan p{{E, routes, topk, K, rows}, blocks > 1 && (int64_t)items * all < 512};
  p.s.cols = std::max(1, std::min({16, 64 / (blocks * terms), (5 * routes + 2 * E - 1) / (2 * E) + 1}));
  p.s.by_route = routes < E;
  const int chunks = std::max(1, (items <= 128 ? 260 : 1200) / items), room = std::max(1, 48 * 1024 / (32 * (K / 32) * ml));
  p.s.pairs = p.split ? 1 : std::min((all + chunks - 1) / chunks, room);
  const int most = items <= 128 ? 16 : 8, turns = (p.s.pairs + most - 1) / most;
  p.s.waves = p.split ? std::min(blocks, 16) : (p.s.pairs + turns - 1) / turns;
  return p;
}

template <bool GU, bool SPLIT, int XT, int ML>
hipError_t run_mm(const MoeShape& sh, const void* src, const int32_t* ids, const uint8_t* bank, const AwqLayout& L, float* dst,
                  hipStream_t st) {
  if (!raise_lds_limit<moe_mm_kernel<GU, SPLIT, XT, ML>>()) return hipErrorInvalidValue;
  const int all = sh.rows / (GU ? 16 : 32);
  hipLaunchKernelGGL((moe_mm_kernel<GU, SPLIT, XT, ML>), dim3((all + sh.pairs - 1) / sh.pairs, std::min(sh.routes, sh.E)),
                     dim3(64 * sh.waves), moe_lds(sh, XT == X_F32 ? 2 : 1, ML, SPLIT).total, st, sh, src, ids, bank, L, dst);
  return hipGetLastError();
}
template <bool GU, int XT, int ML>
hipError_t run_mm(int E, int routes, int topk, int K, int rows, const void* src, const int32_t* ids, const uint8_t* bank,
                  const AwqLayout& L, float* dst, hipStream_t st) {
  const MoePlan p = moe_plan(E, routes, topk, K, rows, GU, XT == X_F32 ? 2 : 1, ML);
  return p.split ? run_mm<GU, true, XT, ML>(p.s, src, ids, bank, L, dst, st) : run_mm<GU, false, XT, ML>(p.s, src, ids, bank, L, dst, st);
}
template <int ML>
hipError_t run_experts(int M, int E, int topk, int H, int I, const void* x, XType xt, const int32_t* ids, const uint8_t* w13,
                       const uint8_t* w2, float* act, float* y, hipStream_t st) {
  const int routes = M * topk;
  const AwqLayout L13 = awq_layout(2 * (int64_t)I, H, ML), L2 = awq_layout(H, I, ML);
  hipError_t e = xt == X_F32    ? run_mm<true, X_F32, ML>(E, routes, topk, H, I, x, ids, w13, L13, act, st)
                 : xt == X_BF16 ? run_mm<true, X_BF16, ML>(E, routes, topk, H, I, x, ids, w13, L13, act, st)
                                : run_mm<true, X_F16, ML>(E, routes, topk, H, I, x, ids, w13, L13, act, st);
  if (e != hipSuccess) return e;
  return run_mm<false, X_F32, ML>(E, routes, topk, I, H, act, ids, w2, L2, y, st);
}
template <int XT, int WT>
void run_logits(int M, int E, int H, const void* x, const void* router, float* logits, hipStream_t st) {
  if (M == 1)
    hipLaunchKernelGGL((route_logits_kernel<XT, WT, 1, 1>), dim3((E + 3) / 4), dim3(256), 0, st, M, E, H, x, router, logits);
  else
    hipLaunchKernelGGL((route_logits_kernel<XT, WT, 2, 4>), dim3((E + 7) / 8, (M + 3) / 4), dim3(256), 0, st, M, E, H, x, router, logits);
}
template <int XT>
void run_logits(int M, int E, int H, const void* x, const void* router, XType rt, float* logits, hipStream_t st) {
  if (rt == X_F32) run_logits<XT, X_F32>(M, E, H, x, router, logits, st);
  else if (rt == X_BF16) run_logits<XT, X_BF16>(M, E, H, x, router, logits, st);
  else run_logits<XT, X_F16>(M, E, H, x, router, logits, st);
}
void run_topk(int M, int E, int topk, int renorm, const float* logits, int32_t* ids, float* weights, hipStream_t st) {
  if (E <= 64) hipLaunchKernelGGL(route_topk_kernel<1>, dim3(M), dim3(64), 0, st, E, topk, renorm, logits, ids, weights);
  else if (E <= 256) hipLaunchKernelGGL(route_topk_kernel<4>, dim3(M), dim3(64), 0, st, E, topk, renorm, logits, ids, weights);
  else if (E <= 512) hipLaunchKernelGGL(route_topk_kernel<8>, dim3(M), dim3(64), 0, st, E, topk, renorm, logits, ids, weights);
  else if (E <= 1024) hipLaunchKernelGGL(route_topk_kernel<16>, dim3(M), dim3(64), 0, st, E, topk, renorm, logits, ids, weights);
  else hipLaunchKernelGGL(route_topk_kernel<0>, dim3(M), dim3(64), 0, st, E, topk, renorm, logits, ids, weights);
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
    run_topk(M, E, topk, renorm ? 1 : 0, logits, ids, weights, st);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  e = meta_layout == 3 ? run_experts<3>(M, E, topk, H, I, x, xt, ids, w13, w2, act, y, st)
                       : run_experts<4>(M, E, topk, H, I, x, xt, ids, w13, w2, act, y, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_sum_kernel, dim3((H + 1023) / 1024, M), dim3(256), 0, st, E, topk, H, ids, weights, y, out, (int)ot);
  return hipGetLastError();
}

}  // namespace wq
