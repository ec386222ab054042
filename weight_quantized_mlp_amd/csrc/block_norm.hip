// Norms before and after a block with its gate and residual (gfx950): block_norm_run and block_norm_backward in
// include/wqmlp_blocks.h.
//
// Rows of H elements, each read once: a workgroup holds its row in registers (chunks of 8 elements per thread) between
// the row sums, so a pass moves the bytes of its inputs and outputs and nothing else.  Rows above 16384 elements (backward: 8192,
// where the columns' sums take registers, too) are read again for every pass instead (they come from L2).  HBM bounds long calls,
// the chain of load, row sum, row sum and store short ones.  Calls in a row: 8191 x 5120 float32 116 us (588 MB, 5.1 TB/s), one
// bfloat16 row of 2560 3.3 us on the device (11 a call, the binding's); backward 4096 x 5120 bfloat16 63 us (252 MB, 4.0 TB/s),
// 129 x 320 float32 8 us on the device in two launches.
//
// Backward, with n = t r the normed row and dn its gradient: dt = r (dn - n mean(dn n)).  Every factor is applied as it stands there; r^3,
// which the mean over t itself would need, leaves float32's range where r and n do not (rows of rms 1e13, or rows of zeros under an eps
// of 1e-26).  The two norms' row sums chain (dy's needs du, which needs the second norm's), while the weights' gradients
// are sums over rows.  A workgroup walks a run of consecutive rows and keeps its columns' three sums in registers; what
// it has at the end goes to the workspace and a second kernel adds the runs in order, so nothing is atomic and the
// result does not depend on timing.  A run never crosses a gate row unless it holds whole gate rows.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "../../include/wqmlp.h"
#include "dev_common.h"
#include "launch.h"

namespace wq {

namespace {

// ---- 8 elements of any type ------------------------------------------------------------------------------------
struct Raw8 { u32x4 a, b; };
// Of a size known at compile time, or at run time: the second load repeats the first one's address for 2-byte types, which is
// cheaper than a branch around a load (the join would wait for it).
template <bool W4>
__device__ __forceinline__ Raw8 load8(const void* p, size_t at) {
  const u32x4* q = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(p) + at * (W4 ? 4 : 2));
  Raw8 r;
  r.a = q[0];
  if constexpr (W4) r.b = q[1];
  else r.b = r.a;
  return r;
}
__device__ __forceinline__ Raw8 load8(const void* p, size_t at, int type) {
  const bool w4 = type == X_F32;
  const u32x4* q = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(p) + (w4 ? at * 4 : at * 2));
  return {q[0], q[w4 ? 1 : 0]};
}
__device__ __forceinline__ void values8(const Raw8& r, int type, float (&v)[8]) {
  if (type == X_F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = r.a[j], b = r.b[j];
      v[j] = __uint_as_float(a);
      v[4 + j] = __uint_as_float(b);
    }
  } else if (type == X_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = r.a[j];
      v[2 * j] = __uint_as_float(a << 16);
      v[2 * j + 1] = __uint_as_float(a & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = r.a[j];
      const f16x2 p = as_f16x2(a);
      v[2 * j] = (float)p.x;
      v[2 * j + 1] = (float)p.y;
    }
  }
}
// Stores 8 floats rounded to the type; v becomes the stored values.
__device__ __forceinline__ void store8(void* p, size_t at, int type, float (&v)[8]) {
  if (type == X_F32) {
    f32x4* q = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + at);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
    return;
  }
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (type == X_BF16) {
      const uint32_t lo = __builtin_bit_cast(uint16_t, (__bf16)v[2 * j]), hi = __builtin_bit_cast(uint16_t, (__bf16)v[2 * j + 1]);
      o[j] = lo | (hi << 16);
      v[2 * j] = __uint_as_float(lo << 16);
      v[2 * j + 1] = __uint_as_float(hi << 16);
    } else {
      const f16x2 h = {(_Float16)v[2 * j], (_Float16)v[2 * j + 1]};
      o[j] = as_u32(h);
      v[2 * j] = (float)h.x;
      v[2 * j + 1] = (float)h.y;
    }
  }
  *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p) + at) = o;
}

// N sums over the workgroup (up to 16 waves), the same in every thread: waves by DPP, then the waves' sums, one per lane of 16, by DPP
// again.  buf alternates between two halves from call to call (`turn`), so that one barrier per call is enough.
constexpr int kMaxWaves = 16;
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* buf, int& turn) {
  float* b = buf + turn * N * kMaxWaves;
  turn ^= 1;
  const int wave = (int)threadIdx.x >> 6, waves = (int)blockDim.x >> 6, lane = (int)threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float s = wave64_sum(v[i]);
    if ((threadIdx.x & 63) == 0) b[i * kMaxWaves + wave] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float s = b[i * kMaxWaves + min(lane, waves - 1)];
    v[i] = row16_sum(lane < waves ? s : 0.f);
  }
}

struct NormArgs {
  int M, H, L;                 // L: rows per gate row
  const void *h, *y, *post, *pre, *gate;
  int ht, yt, xt, wt, gt;
  float alpha, offset, eps;
  bool has_y, has_post, has_pre, has_gate;
};
// Absent vectors read the first row of h as 2-byte elements (which it holds in any type) and are replaced by their neutral value.
__device__ __forceinline__ void weight8(const void* p, bool has, const NormArgs& a, int at, float (&w)[8]) {
  const Raw8 r = load8(has ? p : a.h, at, has ? a.wt : X_BF16);
  values8(r, has ? a.wt : X_BF16, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = has ? w[j] + a.offset : 1.f;
}
__device__ __forceinline__ void gate8(const NormArgs& a, int group, int at, float (&g)[8]) {
  const Raw8 r = load8(a.has_gate ? a.gate : a.h, a.has_gate ? (size_t)group * a.H + at : (size_t)at, a.has_gate ? a.gt : X_BF16);
  values8(r, a.has_gate ? a.gt : X_BF16, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = (a.has_gate ? g[j] : 1.f) * a.alpha;
}

// ---- forward ---------------------------------------------------------------------------------------------------
// A workgroup per row.  A grid dimension holds fewer than 2^32 threads; only 2^23 rows, the most there may be, of 512 threads reach
// that, and go as two halves.  (A row test in the kernel, for any split, costs a short call 0.15 us of 4.)
constexpr int kHalfRows = 1 << 22;
__device__ __forceinline__ int forward_row() { return (int)blockIdx.y * kHalfRows + (int)blockIdx.x; }
inline dim3 forward_grid(int M) { return M == 2 * kHalfRows ? dim3(kHalfRows, 2) : dim3(M); }
static_assert(WQ_MAX_DIM == 2 * kHalfRows, "");
// ho may be a.h itself (in place), so it is not declared restrict; a thread reads its elements of h before it writes them.
template <bool H4, bool Y4, int RC>
__global__ void __launch_bounds__(512) norm_run_kernel(NormArgs a, void* ho, void* __restrict__ xo) {
  __shared__ float buf[2 * kMaxWaves];
  const int C = a.H / 8, T = (int)blockDim.x, t = (int)threadIdx.x, m = forward_row();
  const size_t row = (size_t)m * a.H;
  int turn = 0;
  Raw8 hr[RC], yr[RC];
#pragma unroll
  for (int i = 0; i < RC; ++i) {
    const int c = min(t + i * T, C - 1);
    hr[i] = load8<H4>(a.h, row + 8 * c);
    yr[i] = load8<Y4>(a.y, row + 8 * c);
  }
  float h[RC][8], s[1];
#pragma unroll
  for (int i = 0; i < RC; ++i) values8(hr[i], a.ht, h[i]);
  if (a.has_y) {
    float y[RC][8], r = 1.f;
#pragma unroll
    for (int i = 0; i < RC; ++i) values8(yr[i], a.yt, y[i]);
    if (a.has_post) {
      s[0] = 0.f;
#pragma unroll
      for (int i = 0; i < RC; ++i)
        if (t + i * T < C)
#pragma unroll
          for (int j = 0; j < 8; ++j) s[0] = fmaf(y[i][j], y[i][j], s[0]);
      block_sums(s, buf, turn);
      r = 1.f / sqrtf(s[0] / (float)a.H + a.eps);
    }
    const int group = m / a.L;
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      const int c = min(t + i * T, C - 1);
      float w[8], g[8];
      weight8(a.post, a.has_post, a, 8 * c, w);
      gate8(a, group, 8 * c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = fmaf(g[j], y[i][j] * r * w[j], h[i][j]);
      if (t + i * T < C) store8(ho, row + 8 * c, a.ht, h[i]);
    }
  }
  if (!a.has_pre) return;
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < RC; ++i)
    if (t + i * T < C)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(h[i][j], h[i][j], s[0]);
  block_sums(s, buf, turn);
  const float r = 1.f / sqrtf(s[0] / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < RC; ++i) {
    const int c = min(t + i * T, C - 1);
    float w[8];
    weight8(a.pre, true, a, 8 * c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= h[i][j] * r;
    if (t + i * T < C) store8(xo, row + 8 * c, a.xt, w);
  }
}

// Rows too long to hold: every pass reads them again, each thread the elements that it wrote itself.
__global__ void __launch_bounds__(512) norm_run_long_kernel(NormArgs a, void* ho, void* __restrict__ xo) {
  __shared__ float buf[2 * kMaxWaves];
  const int C = a.H / 8, T = (int)blockDim.x, t = (int)threadIdx.x, m = forward_row();
  const size_t row = (size_t)m * a.H;
  int turn = 0;
  float s[1] = {0.f}, v[8], r = 1.f;
  if (a.has_y) {
    if (a.has_post) {
      for (int c = t; c < C; c += T) {
        values8(load8(a.y, row + 8 * (size_t)c, a.yt), a.yt, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(v[j], v[j], s[0]);
      }
      block_sums(s, buf, turn);
      r = 1.f / sqrtf(s[0] / (float)a.H + a.eps);
    }
    s[0] = 0.f;
    for (int c = t; c < C; c += T) {
      float h[8], w[8], g[8];
      values8(load8(a.h, row + 8 * (size_t)c, a.ht), a.ht, h);
      values8(load8(a.y, row + 8 * (size_t)c, a.yt), a.yt, v);
      weight8(a.post, a.has_post, a, 8 * c, w);
      gate8(a, m / a.L, 8 * c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = fmaf(g[j], v[j] * r * w[j], h[j]);
      store8(ho, row + 8 * (size_t)c, a.ht, h);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(h[j], h[j], s[0]);
    }
  } else {
    for (int c = t; c < C; c += T) {
      values8(load8(a.h, row + 8 * (size_t)c, a.ht), a.ht, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(v[j], v[j], s[0]);
    }
  }
  if (!a.has_pre) return;
  block_sums(s, buf, turn);
  r = 1.f / sqrtf(s[0] / (float)a.H + a.eps);
  const void* src = a.has_y ? ho : a.h;
  for (int c = t; c < C; c += T) {
    float w[8];
    values8(load8(src, row + 8 * (size_t)c, a.ht), a.ht, v);
    weight8(a.pre, true, a, 8 * c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= v[j] * r;
    store8(xo, row + 8 * (size_t)c, a.xt, w);
  }
}

// ---- backward --------------------------------------------------------------------------------------------------
struct GradOut {
  const void *dh, *dx;         // gradients of h_out and x (dh null: zeros)
  void *dhi, *dy;
  float *dpost, *dgate, *dpre; // what the columns' sums go to: the workspace's runs, or the result itself
};
// Runs of consecutive rows.  L >= per: each gate row's L rows in S runs of `per` (the last one shorter); else runs of
// whole gate rows, per / L of them.
struct NormRuns {
  int per, S, runs;
};
// Runs: about one workgroup of ten waves per CU, or as many smaller ones (up to four) as make ten waves: every run costs three rows of
// float32 in the workspace, written and read again.
inline int norm_grad_chunks(int H);              // chunks per thread
inline int norm_grad_threads(int H);
inline NormRuns norm_runs(int M, int H, int G) {
  const int L = M / G, runs = 256 * std::max(1, std::min(4, 640 / norm_grad_threads(H)));
  NormRuns p;
  const int want = std::max(1, (M + runs - 1) / runs);
  if (L >= want) {
    p.S = (L + want - 1) / want;
    p.per = (L + p.S - 1) / p.S;
    p.S = (L + p.per - 1) / p.per;
    p.runs = G * p.S;
  } else {
    p.S = 1;
    p.per = (want + L - 1) / L * L;
    p.runs = (M + p.per - 1) / p.per;
  }
  return p;
}
// First and last row of run b.
__device__ __forceinline__ void run_rows(const NormRuns& p, int M, int L, int b, int& r0, int& r1) {
  if (p.per < L || p.S > 1) {
    const int g = b / p.S, s = b - g * p.S;
    r0 = g * L + s * p.per;
    r1 = min(r0 + p.per, (g + 1) * L);
  } else {
    r0 = b * p.per;
    r1 = min(r0 + p.per, M);
  }
}

struct RowScalars {
  float ru, rv, cu;            // r(h), r(y) (1 without post), mean(dn n(h))
};
// du of one element; what is absent takes no part, whatever stands in its place.
__device__ __forceinline__ float norm_du(bool has_pre, bool has_dh, float ru, float cu, float dn, float h, float dh) {
  const float past = has_dh ? dh : 0.f;
  return has_pre ? fmaf(ru, fmaf(-cu, h * ru, dn), past) : past;
}

// Rows in registers.  Of one chunk per thread the next row's loads are on their way while this one's sums are formed; the weights and
// the gate row (until it changes) stay in registers.  One workgroup fills a CU, so a row's operations stand in its chain beside the two
// row sums, with nothing else to run meanwhile (spread evenly over all lanes they are 13 us of the 63): what is absent is zeroed once instead of selected,
// and the decoding of 2-byte tensors does not branch where all of them are bfloat16 (BF; 4096 x 2560: 57 us without either, 36).
template <bool W4, bool BF>
__device__ __forceinline__ void row_values(const Raw8& r, int type, float (&v)[8]) {
  if constexpr (W4) values8(r, X_F32, v);
  else if constexpr (BF) values8(r, X_BF16, v);
  else values8(r, type == X_BF16 ? X_BF16 : X_F16, v);
}
template <bool W4, bool BF>
__device__ __forceinline__ void row_store(void* p, size_t at, int type, float (&v)[8]) {
  if constexpr (W4) store8(p, at, X_F32, v);
  else if constexpr (BF) store8(p, at, X_BF16, v);
  else store8(p, at, type == X_BF16 ? X_BF16 : X_F16, v);
}

template <bool H4, bool Y4, bool X4, bool BF, int RC>
__global__ void __launch_bounds__(RC == 1 ? 640 : 512) norm_grad_kernel(NormArgs a, NormRuns p, GradOut o) {
  __shared__ float buf2[2 * 3 * kMaxWaves], buf1[2 * kMaxWaves];
  constexpr bool AHEAD = RC == 1;                 // (two chunks of two rows spill)
  const int C = a.H / 8, T = (int)blockDim.x, t = (int)threadIdx.x, b = (int)blockIdx.x;
  const bool has_dh = o.dh != nullptr;
  const void* dhp = has_dh ? o.dh : a.h;
  int r0, r1, turn2 = 0, turn1 = 0;
  run_rows(p, a.M, a.L, b, r0, r1);
  Raw8 hr[RC], yr[RC], dhr[RC], dxr[RC];
  float pre[RC][8], post[RC][8], gate[RC][8];
  int at[RC];
#pragma unroll
  for (int i = 0; i < RC; ++i) {
    at[i] = 8 * min(t + i * T, C - 1);
    weight8(a.pre, a.has_pre, a, at[i], pre[i]);
    weight8(a.post, a.has_post, a, at[i], post[i]);
  }
  auto load_gate = [&](int m) {
#pragma unroll
    for (int i = 0; i < RC; ++i) gate8(a, m / a.L, at[i], gate[i]);   // with alpha
  };
  auto load_row = [&](int m) {
    const size_t row = (size_t)m * a.H;
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      hr[i] = load8<H4>(a.h, row + at[i]);
      yr[i] = load8<Y4>(a.y, row + at[i]);
      dhr[i] = load8<H4>(dhp, row + at[i]);
      dxr[i] = load8<X4>(o.dx, row + at[i]);
    }
  };
  float spre[RC][8], spost[RC][8], sgate[RC][8];
#pragma unroll
  for (int i = 0; i < RC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) spre[i][j] = spost[i][j] = sgate[i][j] = 0.f;
  const float invH = 1.f / (float)a.H;
  int left = a.L - r0 % a.L;                      // rows of the gate row from this one on
  if (r0 < r1) {
    load_gate(r0);
    if (AHEAD) load_row(r0);
  }
  for (int m = r0; m < r1; ++m) {
    const size_t row = (size_t)m * a.H;
    if (!AHEAD) load_row(m);
    float h[RC][8], y[RC][8], dh[RC][8], dx[RC][8], s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      row_values<H4, BF>(hr[i], a.ht, h[i]);
      row_values<Y4, BF>(yr[i], a.yt, y[i]);
      row_values<H4, BF>(dhr[i], a.ht, dh[i]);
      row_values<X4, BF>(dxr[i], a.xt, dx[i]);
    }
    if (!a.has_pre)
#pragma unroll
      for (int i = 0; i < RC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = dx[i][j] = 0.f;
    if (!has_dh)
#pragma unroll
      for (int i = 0; i < RC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dh[i][j] = 0.f;
#pragma unroll
    for (int i = 0; i < RC; ++i)
      if (t + i * T < C)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[0] = fmaf(h[i][j], h[i][j], s[0]);
          s[1] = fmaf(dx[i][j] * pre[i][j], h[i][j], s[1]);
          s[2] = fmaf(y[i][j], y[i][j], s[2]);
        }
    if (AHEAD && m + 1 < r1) load_row(m + 1);
    block_sums(s, buf2, turn2);
    const float ru = a.has_pre ? 1.f / sqrtf(s[0] * invH + a.eps) : 0.f;
    const float cu = a.has_pre ? -(s[1] * invH) * ru : 0.f;   // -mean(dn n(h))
    const float rv = a.has_post ? 1.f / sqrtf(s[2] * invH + a.eps) : 1.f;
    float q[1] = {0.f};                           // dx becomes dp: alpha gate du post+
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      if (t + i * T >= C) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hn = h[i][j] * ru, du = fmaf(ru, fmaf(cu, hn, dx[i][j] * pre[i][j]), dh[i][j]);
        dh[i][j] = du;
        spre[i][j] = fmaf(dx[i][j], hn, spre[i][j]);
        const float n = y[i][j] * rv, dg = gate[i][j] * du;              // n(y), or y
        y[i][j] = n;
        spost[i][j] = fmaf(dg, n, spost[i][j]);
        sgate[i][j] = fmaf(du, n * post[i][j], sgate[i][j]);             // times alpha at the end
        dx[i][j] = dg * post[i][j];
        q[0] = fmaf(dx[i][j], n, q[0]);
      }
      if (o.dhi != nullptr) row_store<H4, BF>(o.dhi, row + at[i], a.ht, dh[i]);
    }
    if (o.dy != nullptr) {
      if (a.has_post) {
        block_sums(q, buf1, turn1);
        const float cy = -q[0] * invH;            // -mean(dp post+ n(y))
#pragma unroll
        for (int i = 0; i < RC; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) dx[i][j] = rv * fmaf(cy, y[i][j], dx[i][j]);
      }
#pragma unroll
      for (int i = 0; i < RC; ++i)
        if (t + i * T < C) row_store<Y4, BF>(o.dy, row + at[i], a.yt, dx[i]);
    }
    if (--left == 0) {
      left = a.L;
      // the gate row's sums, where a run holds whole gate rows and this was its last row
      if (o.dgate != nullptr && p.S == 1) {
#pragma unroll
        for (int i = 0; i < RC; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) sgate[i][j] *= a.alpha;
          if (t + i * T < C) store8(o.dgate, (size_t)(m / a.L) * a.H + at[i], X_F32, sgate[i]);
#pragma unroll
          for (int j = 0; j < 8; ++j) sgate[i][j] = 0.f;
        }
      }
      if (m + 1 < r1) load_gate(m + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < RC; ++i) {
    if (t + i * T >= C) continue;
    const size_t to = (size_t)b * a.H + at[i];
#pragma unroll
    for (int j = 0; j < 8; ++j) sgate[i][j] *= a.alpha;
    if (o.dpre != nullptr) store8(o.dpre, to, X_F32, spre[i]);
    if (o.dpost != nullptr) store8(o.dpost, to, X_F32, spost[i]);
    if (o.dgate != nullptr && p.S > 1) store8(o.dgate, to, X_F32, sgate[i]);
  }
}

// Rows too long to hold.  A workgroup per row: dy and the row's scalars; dh_in and the columns' sums follow in
// norm_grad_cols_kernel, from the inputs again, so that dh_in may stand where dh does.
__global__ void __launch_bounds__(512) norm_grad_long_kernel(NormArgs a, GradOut o, RowScalars* __restrict__ rows) {
  __shared__ float buf2[2 * 3 * kMaxWaves], buf1[2 * kMaxWaves];
  const int C = a.H / 8, T = (int)blockDim.x, t = (int)threadIdx.x, m = (int)blockIdx.x;
  const bool has_dh = o.dh != nullptr;
  const size_t row = (size_t)m * a.H;
  int turn2 = 0, turn1 = 0;
  const float invH = 1.f / (float)a.H;
  float s[3] = {0.f, 0.f, 0.f}, h[8], y[8], dh[8], dx[8], w[8], v[8], g[8];
  for (int c = t; c < C; c += T) {
    const size_t at = row + 8 * (size_t)c;
    values8(load8(a.h, at, a.ht), a.ht, h);
    values8(load8(a.y, at, a.yt), a.yt, y);
    values8(load8(o.dx, at, a.xt), a.xt, dx);
    weight8(a.pre, a.has_pre, a, 8 * c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[0] = fmaf(h[j], h[j], s[0]);
      s[1] = fmaf(dx[j] * w[j], h[j], s[1]);
      s[2] = fmaf(y[j], y[j], s[2]);
    }
  }
  block_sums(s, buf2, turn2);
  const float ru = a.has_pre ? 1.f / sqrtf(s[0] * invH + a.eps) : 0.f;
  const float cu = a.has_pre ? s[1] * invH * ru : 0.f;
  const float rv = a.has_post ? 1.f / sqrtf(s[2] * invH + a.eps) : 1.f;
  if (t == 0) rows[m] = {ru, rv, cu};
  auto du8 = [&](int c) {                         // dh becomes du, w and v the weights, g the gate with alpha
    const size_t at = row + 8 * (size_t)c;
    values8(load8(a.h, at, a.ht), a.ht, h);
    values8(load8(a.y, at, a.yt), a.yt, y);
    values8(load8(has_dh ? o.dh : a.h, at, a.ht), a.ht, dh);
    values8(load8(o.dx, at, a.xt), a.xt, dx);
    weight8(a.pre, a.has_pre, a, 8 * c, w);
    weight8(a.post, a.has_post, a, 8 * c, v);
    gate8(a, m / a.L, 8 * c, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) dh[j] = norm_du(a.has_pre, has_dh, ru, cu, dx[j] * w[j], h[j], dh[j]);
  };
  float cy = 0.f;
  if (o.dy != nullptr && a.has_post) {
    float q[1] = {0.f};
    for (int c = t; c < C; c += T) {
      du8(c);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[0] = fmaf(g[j] * dh[j] * v[j], y[j] * rv, q[0]);
    }
    block_sums(q, buf1, turn1);
    cy = q[0] * invH;
  }
  if (o.dy != nullptr) {
    for (int c = t; c < C; c += T) {
      du8(c);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = a.has_post ? rv * fmaf(-cy, y[j] * rv, g[j] * dh[j] * v[j]) : g[j] * dh[j];
      store8(o.dy, row + 8 * (size_t)c, a.yt, y);
    }
  }
}
// du of a row again, from the stored scalars: a thread's 8 columns over the rows of a run; then, where asked for, dh_in (last,
// since it may stand where dh does).
__global__ void __launch_bounds__(64) norm_grad_cols_kernel(NormArgs a, NormRuns p, GradOut o, const RowScalars* __restrict__ rows) {
  const int C = a.H / 8, c = (int)(blockIdx.x * 64 + threadIdx.x), b = (int)blockIdx.y;
  if (c >= C) return;
  const bool has_dh = o.dh != nullptr;
  int r0, r1;
  run_rows(p, a.M, a.L, b, r0, r1);
  float spre[8] = {}, spost[8] = {}, sgate[8] = {}, h[8], y[8], dh[8], dx[8], w[8], v[8], g[8];
  weight8(a.pre, a.has_pre, a, 8 * c, w);
  weight8(a.post, a.has_post, a, 8 * c, v);
  for (int m = r0; m < r1; ++m) {
    const size_t at = (size_t)m * a.H + 8 * (size_t)c;
    const RowScalars k = rows[m];
    values8(load8(a.h, at, a.ht), a.ht, h);
    values8(load8(a.y, at, a.yt), a.yt, y);
    values8(load8(has_dh ? o.dh : a.h, at, a.ht), a.ht, dh);
    values8(load8(o.dx, at, a.xt), a.xt, dx);
    gate8(a, m / a.L, 8 * c, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float du = norm_du(a.has_pre, has_dh, k.ru, k.cu, dx[j] * w[j], h[j], dh[j]);
      const float n = y[j] * k.rv;
      spre[j] = fmaf(dx[j], h[j] * k.ru, spre[j]);
      spost[j] = fmaf(g[j] * du, n, spost[j]);
      sgate[j] = fmaf(a.alpha * du, n * v[j], sgate[j]);
      dh[j] = du;
    }
    if (o.dhi != nullptr) store8(o.dhi, at, a.ht, dh);
    if (o.dgate != nullptr && p.S == 1 && (m + 1) % a.L == 0) {
      store8(o.dgate, (size_t)(m / a.L) * a.H + 8 * c, X_F32, sgate);
#pragma unroll
      for (int j = 0; j < 8; ++j) sgate[j] = 0.f;
    }
  }
  const size_t at = (size_t)b * a.H + 8 * (size_t)c;
  if (o.dpre != nullptr) store8(o.dpre, at, X_F32, spre);
  if (o.dpost != nullptr) store8(o.dpost, at, X_F32, spost);
  if (o.dgate != nullptr && p.S > 1) store8(o.dgate, at, X_F32, sgate);
}

// Sums of the runs, in order: thread (column, lane of 32) adds every 32nd run, then the 32 lanes' sums in pairs, 16
// apart, then 8, ... (five roundings in a chain instead of 31).  blockIdx.y: dpre, dpost, then the gate rows, each over its own S runs.
struct NormJoin {
  const float* src[3];
  float* dst[3];               // dpre, dpost, dgate (null: none)
  int n, S, G;                 // n: runs; S, G as in NormRuns
};
__global__ void __launch_bounds__(1024) norm_join_kernel(int H, NormJoin j) {
  __shared__ float part[32][33];
  const int col = (int)threadIdx.x & 31, k = (int)threadIdx.x >> 5, at = (int)blockIdx.x * 32 + col;
  const int z = (int)blockIdx.y;
  const int which = z < 2 ? z : 2;
  const float* src = j.src[which];
  float* dst = j.dst[which];
  if (dst == nullptr) return;
  int n = j.n;
  if (which == 2) {
    src += (size_t)(z - 2) * j.S * H;
    dst += (size_t)(z - 2) * H;
    n = j.S;
  }
  float s = 0.f;
  if (at < H)
    for (int r = k; r < n; r += 32) s += src[(size_t)r * H + at];
  part[k][col] = s;
  __syncthreads();
  if (k == 0 && at < H) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = part[i][col];
#pragma unroll
    for (int half = 16; half >= 1; half >>= 1)
#pragma unroll
      for (int i = 0; i < half; ++i) v[i] += v[i + half];
    dst[at] = v[0];
  }
}
// (At most kZeroGrid workgroups: a gradient of gate rows may have more elements than a grid dimension holds threads.)
constexpr size_t kZeroGrid = 1 << 20;
__global__ void __launch_bounds__(256) norm_zero_kernel(float* __restrict__ p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = 0.f;
}

inline int threads_for(int C, int rc) { return ((C + rc - 1) / rc + 63) / 64 * 64; }
// Chunks per thread (0: too long to hold).  Forward: at most 512 threads of up to 4 chunks.  Backward: one chunk for up to 640 threads, else
// two for up to 512 (four spill).
inline int held_chunks(int H) {
  const int C = H / 8;
  return C <= 512 ? 1 : (C <= 1024 ? 2 : (C <= 2048 ? 4 : 0));
}
inline int norm_grad_chunks(int H) {
  const int C = H / 8;
  return C <= 640 ? 1 : (C <= 1024 ? 2 : 0);
}
inline int norm_grad_threads(int H) {
  const int rc = norm_grad_chunks(H);
  return rc == 0 ? 512 : threads_for(H / 8, rc);
}

// Workspace of the backward pass: the runs' sums for dpre, dpost, dgate, then the rows' scalars of long rows.
struct NormWs {
  size_t sums, rows, total;
};
inline NormWs norm_ws(int M, int H, int G) {
  const NormRuns p = norm_runs(M, H, G);
  NormWs w;
  w.sums = align256((size_t)p.runs * H * 4);
  w.rows = 3 * w.sums;
  w.total = w.rows + (norm_grad_chunks(H) == 0 ? align256((size_t)M * sizeof(RowScalars)) : 0);
  return w;
}

}  // namespace

hipError_t launch_block_norm(int M, int H, const BlockNorm& n, void* h_out, void* x, XType xt, hipStream_t st) {
  NormArgs a{M, H, M / n.G, n.h, n.y, n.post, n.pre, n.gate, n.ht, n.yt, xt, n.wt, n.gt, n.alpha, n.offset, n.eps,
             n.y != nullptr, n.post != nullptr, n.pre != nullptr, n.gate != nullptr};
  if (!a.has_y) a.y = a.h, a.yt = a.ht;
  const int rc = held_chunks(H);
  if (rc == 0) {
    hipLaunchKernelGGL(norm_run_long_kernel, forward_grid(M), dim3(512), 0, st, a, h_out, x);
    return hipGetLastError();
  }
  const int T = threads_for(H / 8, rc);
  auto go = [&](auto h4, auto y4, auto c) {
    hipLaunchKernelGGL((norm_run_kernel<decltype(h4)::value, decltype(y4)::value, decltype(c)::value>), forward_grid(M), dim3(T),
                       0, st, a, h_out, x);
  };
  auto by_rc = [&](auto h4, auto y4) {
    if (rc == 1) go(h4, y4, std::integral_constant<int, 1>{});
    else if (rc == 2) go(h4, y4, std::integral_constant<int, 2>{});
    else go(h4, y4, std::integral_constant<int, 4>{});
  };
  if (a.ht == X_F32) a.yt == X_F32 ? by_rc(std::true_type{}, std::true_type{}) : by_rc(std::true_type{}, std::false_type{});
  else a.yt == X_F32 ? by_rc(std::false_type{}, std::true_type{}) : by_rc(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

size_t block_norm_grad_scratch_bytes(int M, int H, int G) { return M == 0 ? 0 : norm_ws(M, H, G).total; }

hipError_t launch_block_norm_grad(int M, int H, const BlockNorm& n, const void* dh, const void* dx, XType xt, void* ws,
                                  void* dh_in, void* dy, float* dpost, float* dgate, float* dpre, hipStream_t st) {
  if (M == 0) {
    const std::pair<float*, size_t> zeros[3] = {{dpost, (size_t)H}, {dgate, (size_t)n.G * H}, {dpre, (size_t)H}};
    for (auto [p, count] : zeros) {
      if (p == nullptr || count == 0) continue;
      hipLaunchKernelGGL(norm_zero_kernel, dim3((unsigned)std::min((count + 255) / 256, kZeroGrid)), dim3(256), 0, st, p, count);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  NormArgs a{M, H, M / n.G, n.h, n.y, n.post, n.pre, n.gate, n.ht, n.yt, xt, n.wt, n.gt, n.alpha, n.offset, n.eps,
             n.y != nullptr, n.post != nullptr, n.pre != nullptr, n.gate != nullptr};
  if (!a.has_y) a.y = a.h, a.yt = a.ht;
  if (!a.has_pre) dx = a.h, a.xt = a.ht;
  const NormRuns p = norm_runs(M, H, n.G);
  const NormWs L = norm_ws(M, H, n.G);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  auto runs = [&](int i) { return reinterpret_cast<float*>(base + i * L.sums); };
  GradOut o{dh, dx, dh_in, dy, dpost ? runs(1) : nullptr, dgate ? (p.S > 1 ? runs(2) : dgate) : nullptr, dpre ? runs(0) : nullptr};
  const int rc = norm_grad_chunks(H);
  if (rc == 0) {
    RowScalars* rows = reinterpret_cast<RowScalars*>(base + L.rows);
    hipLaunchKernelGGL(norm_grad_long_kernel, dim3(M), dim3(512), 0, st, a, o, rows);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(norm_grad_cols_kernel, dim3((H / 8 + 63) / 64, p.runs), dim3(64), 0, st, a, p, o, rows);
  } else {
    const int T = norm_grad_threads(H);
    const bool bf = a.ht != X_F16 && a.yt != X_F16 && a.xt != X_F16;
    auto go = [&](auto h4, auto y4, auto x4, auto bfs, auto c) {
      hipLaunchKernelGGL((norm_grad_kernel<decltype(h4)::value, decltype(y4)::value, decltype(x4)::value, decltype(bfs)::value,
                                           decltype(c)::value>),
                         dim3(p.runs), dim3(T), 0, st, a, p, o);
    };
    auto by_bf = [&](auto h4, auto y4, auto x4, auto c) { bf ? go(h4, y4, x4, std::true_type{}, c) : go(h4, y4, x4, std::false_type{}, c); };
    auto by_rc = [&](auto h4, auto y4, auto x4) {
      if (rc == 1) by_bf(h4, y4, x4, std::integral_constant<int, 1>{});
      else by_bf(h4, y4, x4, std::integral_constant<int, 2>{});
    };
    auto by_x = [&](auto h4, auto y4) { a.xt == X_F32 ? by_rc(h4, y4, std::true_type{}) : by_rc(h4, y4, std::false_type{}); };
    auto by_y = [&](auto h4) { a.yt == X_F32 ? by_x(h4, std::true_type{}) : by_x(h4, std::false_type{}); };
    a.ht == X_F32 ? by_y(std::true_type{}) : by_y(std::false_type{});
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool join_gate = dgate != nullptr && p.S > 1;
  if (dpost == nullptr && dpre == nullptr && !join_gate) return hipSuccess;
  NormJoin j{{runs(0), runs(1), runs(2)}, {dpre, dpost, join_gate ? dgate : nullptr}, p.runs, p.S, n.G};
  hipLaunchKernelGGL(norm_join_kernel, dim3((H + 31) / 32, 2 + (join_gate ? n.G : 0)), dim3(1024), 0, st, H, j);
  return hipGetLastError();
}

}  // namespace wq
