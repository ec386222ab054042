// Low-rank adapters, the weight gradients (gfx950): g[e][r,d] = sum over the rows m of adapter e of t[m,r] v[m,d]
// (db from t = scale x a^T and v = dy, da from t = scale dy b and v = x).
//
// v is the bytes, read once per adapter that a block of rows names.  A workgroup owns one adapter, 64 columns d and
// up to 64 ranks; its 4 waves (or its one, see outer_one_wave) take blocks of 32 rows in turn, each with its own accumulators, so
// no barrier stands between blocks, and add them through LDS at the end.  Which blocks hold rows of the adapter is found first, from
// the ids, as one 32-bit mask per block; other blocks are never loaded, and rows of other adapters enter as zeros
// (in v as well, so that nothing a foreign row holds can reach the sum).  Both operands have the contraction (rows)
// as their slow index, so both go through the wave's transposing LDS tiles, t's three terms one after the other through
// the same one (a tile per term left room for two workgroups on a CU at rank 32, one at rank 64); the next block's loads
// are issued before this block's MFMAs.  Long batches with few adapters split the rows over up to 8 workgroups, joined in
// order by a second kernel.  da and db of a backward pass share a launch where x and dy have one type and both take as many waves,
// and always the second kernel's.  Shortest and mean of 20 calls: 4096 x 17408 float32 (db,
// rank 16) 62 and 66 us (4.3-4.6 TB/s); da and db of 2047 x (17408 + 5120) bfloat16, rank 32 on 5 adapters 32 and 34 us, and 31
// with all operands cached: its 2112 short workgroups bound it, not memory.
#include <algorithm>

#include "lora_common.h"

namespace wq {

namespace {

using namespace lora;

constexpr int kD = 64;               // columns of a workgroup
constexpr int kScan = 4096;          // rows whose masks are held at once
constexpr int kParts = 8;            // most parts of the rows

// A wave's LDS: a block of v and of t's terms.  16-bit v is held as transposing term planes; float32 v as it is (padded rows),
// and a lane gathers its 8 rows of a column by 4-byte reads, which needs less room than three planes.
constexpr int kVRow = kD * 4 + 16;
template <int VT> constexpr int outer_v_lds() { return VT == X_F32 ? kRows * kVRow : terms<VT>() * tr_plane<kD>(); }
template <int VT, int NR> constexpr int outer_wave_lds() { return outer_v_lds<VT>() + tr_plane<16 * NR>(); }
template <int VT, int NR, int WAVES> constexpr int outer_lds() {
  const int stage = WAVES * outer_wave_lds<VT, NR>(), red = WAVES == 1 ? 0 : WAVES * 16 * kD * 4;
  return stage > red ? stage : red;
}

// Rows of one workgroup's part: a multiple of kRows.
inline int outer_part_rows(int M, int parts) { return ((M + parts - 1) / parts + kRows - 1) / kRows * kRows; }

// A 16-byte piece without its first s elements, zeros behind the rest (s beyond the piece: of a piece of zeros).
template <int VT>
__device__ __forceinline__ u32x4 drop_first(u32x4 v, int s) {
  constexpr int D2 = VT == X_F32 ? 2 : 4, D1 = D2 / 2;    // elements of two dwords, of one
  if (s & D2) v = u32x4{v.z, v.w, 0u, 0u};
  if (s & D1) v = u32x4{v.y, v.z, v.w, 0u};
  if constexpr (VT != X_F32) {
    if (s & 1)
      v = u32x4{v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16};
  }
  return v;
}

// One of a launch's sums: its operands, the workgroups of its (columns, rank chunks, parts, adapters) and where they write
// (g itself, or the parts' arrays one after the other).
struct OuterSum {
  const uint16_t* t;
  const uint8_t* v;
  float* g;
  int wgs, D, parts, part_rows;
  bool rcontig;                      // g's rank index is contiguous, else its columns are
};

template <int VT, int NR, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) lora_outer_kernel(int M, int E, int R, int total, OuterSum first, OuterSum second,
                                                         const int32_t* __restrict__ ids) {
  constexpr int C = 16 * NR, NV = terms<VT>(), J = kD / 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ uint32_t masks[kScan / kRows];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, gr = lane >> 4;
  const int RC = (R + C - 1) / C;
  uint8_t* vt = lds + wave * outer_wave_lds<VT, NR>();
  uint8_t* ut = vt + outer_v_lds<VT>();
  for (int wg = blockIdx.x; wg < total; wg += gridDim.x) {
    const bool two = wg >= first.wgs;
    const uint16_t* t = two ? second.t : first.t;
    const uint8_t* v = two ? second.v : first.v;
    const int D = two ? second.D : first.D, parts = two ? second.parts : first.parts;
    // columns fastest, then rank chunks, parts and adapters; in 32 bits (three 64-bit divisions were 450 instructions)
    const int w0 = two ? wg - first.wgs : wg, nd = (D + kD - 1) / kD, w1 = w0 / nd, w2 = w1 / RC;
    const int d0 = (w0 - w1 * nd) * kD, r0 = (w1 - w2 * RC) * C, e = w2 / parts, part = w2 - e * parts;
    const int part_rows = two ? second.part_rows : first.part_rows;
    const int mb = part * part_rows, me = min(mb + part_rows, M);
    f32x4 acc[NR][J];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = mb; s0 < me; s0 += kScan) {
      __syncthreads();                                  // the masks' and the tiles' last readers
      const int groups = (min(kScan, me - s0) + 63) / 64;
      for (int i0 = wave; i0 < groups; i0 += 8 * WAVES) {   // 8 groups of 64 rows in flight per wave
        int id[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) id[q] = ids[min(s0 + 64 * (i0 + WAVES * q) + lane, me - 1)];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int i = i0 + WAVES * q;
          const uint64_t b = __ballot(s0 + 64 * i + lane < me && id[q] == e);
          if (lane < 2 && i < groups) masks[2 * i + lane] = (uint32_t)(b >> (32 * lane));
        }
      }
      __syncthreads();
      const int blocks = (min(kScan, me - s0) + kRows - 1) / kRows;
      auto next = [&](int b) {
        while (b < blocks && masks[b] == 0) b += WAVES;
        return b;
      };
      // one block's loads, in whole lines: 16-byte pieces of v, chunks of 8 ranks of each term of t
      constexpr int VP = 16 / esize<VT>(), VL = kD / VP, VN = kRows * VL / 64;   // 16-byte pieces of v: elements, per row, per lane
      u32x4 raw[VN];
      u32x4 u[3][NR];
      // a lane's pieces are of one column; the one that the rows' end cuts is loaded further left, whole, and shifted into place
      const int dv = d0 + VP * (lane % VL), dl = max(min(dv, D - VP), 0), cut = D >= VP ? dv - dl : 0;
      auto load_v = [&](int b) {
        const uint32_t mask = masks[b];
        const int m0 = s0 + kRows * b;
        if (D >= VP) {                                    // the same for all lanes: no branch between the loads
#pragma unroll
          for (int q = 0; q < VN; ++q) {
            const int row = (lane + 64 * q) / VL;
            const uint8_t* p = v + ((size_t)(m0 + row) * D + dl) * esize<VT>();
            raw[q] = u32x4{0u, 0u, 0u, 0u};
            if ((mask >> row & 1) && dv < D) {
              if constexpr (VT == X_F32) raw[q] = *reinterpret_cast<const u32x4_a4*>(p);
              else raw[q] = *reinterpret_cast<const u32x4_a2*>(p);
            }
          }
        } else {                                          // a row is less than a piece
#pragma unroll
          for (int q = 0; q < VN; ++q) {
            const int row = (lane + 64 * q) / VL;
            raw[q] = u32x4{0u, 0u, 0u, 0u};
            if (!(mask >> row & 1) || dv > 0) continue;
            Raw<VT> part;
            raw_load_part<VT>(v + (size_t)(m0 + row) * D * esize<VT>(), D, part);
            raw[q] = part.v[0];
          }
        }
      };
      auto load_u = [&](int b) {
        const uint32_t mask = masks[b];
        const int m0 = s0 + kRows * b;
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          const int c = lane + 64 * q, row = c / (C / 8), r = r0 + 8 * (c % (C / 8));
          const bool on = (mask >> row & 1) != 0 && r < R;
          const uint16_t* p = t + (size_t)(m0 + row) * R + r;
#pragma unroll
          for (int i = 0; i < 3; ++i)
            u[i][q] = on ? *reinterpret_cast<const u32x4*>(p + i * (size_t)M * R) : u32x4{0u, 0u, 0u, 0u};
        }
      };
      auto put_u = [&](int i, const u32x4 (&v)[NR]) {    // term i of t
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          const int c = lane + 64 * q;
          *reinterpret_cast<u32x4*>(ut + (c / (C / 8)) * tr_stride<C>() + (c % (C / 8)) * 16) = v[q];
        }
      };
      int b = next(wave);
      if (b < blocks) load_v(b), load_u(b);
      while (b < blocks) {
        if (d0 + kD > D) {
#pragma unroll
          for (int q = 0; q < VN; ++q) raw[q] = drop_first<VT>(raw[q], cut);
        }
        wave_lds_fence();
#pragma unroll
        for (int q = 0; q < VN; ++q) {
          const int c = lane + 64 * q;
          if constexpr (VT == X_F32) *reinterpret_cast<u32x4*>(vt + (c / VL) * kVRow + (c % VL) * 16) = raw[q];
          else tr_write<VT, kD>(vt, c, Raw<VT>{{raw[q]}});
        }
        put_u(2, u[2]);
        wave_lds_fence();
        b = next(b + WAVES);
        if (b < blocks) load_v(b);
        bf16x8 vf[J][NV];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if constexpr (VT == X_F32) {
            float x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = *reinterpret_cast<const float*>(vt + (8 * gr + q) * kVRow + (16 * j + l16) * 4);
            split3<8>(x, vf[j]);
          } else {
            tr_read<kD, NV>(vt, j, vf[j]);
          }
        }
        u32x4 u1[NR], u0[NR];
#pragma unroll
        for (int q = 0; q < NR; ++q) u1[q] = u[1][q], u0[q] = u[0][q];
        if (b < blocks) load_u(b);
#pragma unroll
        for (int i = 2; i >= 0; --i) {
          if (i < 2) {
            wave_lds_fence();
            put_u(i, i == 1 ? u1 : u0);
            wave_lds_fence();
          }
          bf16x8 uf[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) tr_read<C, 1>(ut, r, &uf[r]);
#pragma unroll
          for (int j = 0; j < J; ++j)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
              for (int k = NV - 1; k >= 0; --k)           // small products first
                if (i + k <= 2) acc[r][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(uf[r], vf[j][k], acc[r][j], 0, 0, 0);
        }
      }
    }

    // fragment (i, j), lane: ranks 16 i + 4 gr .. + 3 of column 16 j + l16
    float* ge = (two ? second.g : first.g) + ((size_t)part * E + e) * (size_t)R * D;
    const bool rcontig = two ? second.rcontig : first.rcontig;
    auto store = [&](int i, int j, f32x4 s) {
      const int d = d0 + 16 * j + l16, r = r0 + 16 * i + 4 * gr;
      if (d >= D || r >= R) return;                       // R is a multiple of 8
      if (rcontig) {
        *reinterpret_cast<f32x4*>(ge + (size_t)d * R + r) = s;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) ge[(size_t)(r + q) * D + d] = s[q];
      }
    };
    if constexpr (WAVES == 1) {
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) store(i, j, acc[i][j]);
    } else {                                              // the four waves' sums in wave order, 16 ranks at a time
      f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) red[(wave * J + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        f32x4 s = red[wave * 64 + lane];
#pragma unroll
        for (int q = 1; q < 4; ++q) s += red[(q * J + wave) * 64 + lane];
        store(i, wave, s);
      }
    }
    __syncthreads();
  }
}

// out[i] = the sum of `parts` arrays of 4 n4 float32, in order; two such sums, the second behind the first.
struct JoinSum {
  const f32x4* p;
  f32x4* out;
  int64_t n4;
  int parts;
};
__global__ void __launch_bounds__(256) lora_join_kernel(JoinSum a, JoinSum b) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.n4 + b.n4; i += (int64_t)gridDim.x * 256) {
    const bool two = i >= a.n4;
    const int64_t at = two ? i - a.n4 : i, n4 = two ? b.n4 : a.n4;
    const f32x4* p = two ? b.p : a.p;
    const int parts = two ? b.parts : a.parts;
    f32x4 v[kParts];                       // all loads in flight together
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      if (q < parts) v[q] = p[(int64_t)q * n4 + at];
    f32x4 s = v[0];
#pragma unroll
    for (int q = 1; q < kParts; ++q)
      if (q < parts) s += v[q];
    (two ? b.out : a.out)[at] = s;
  }
}

inline int64_t outer_tiles(int D, int E, int R) {
  const int C = R <= 16 ? 16 : (R <= 32 ? 32 : 64);
  return (int64_t)E * ((D + kD - 1) / kD) * ((R + C - 1) / C);
}
// Parts of the rows: the number, at most 8 and of at least 256 rows each, for which reading v (stretched by the last round of
// workgroups standing partly idle), the partial sums' way through memory and what a workgroup's start and end cost (about 5 us
// of its share of the bandwidth, 28 KB) take the fewest bytes.  A round is taken as 768 workgroups, 3 per CU, for every form;
// their registers let 4 stand on one (bfloat16 up to rank 16), 3 (bfloat16 up to rank 32, float16 up to 16), 2, or 1 (float32
// above rank 32).  Rounds of 512, 768 and 1024, da and db of a call: 4096 rows of 4096 x 4096, rank 128, float32 dy 145, 164 and
// 157 us; 4096 rows of 5120 x 5120 bfloat16, rank 64 on 4 adapters 97, 89 and 94; 2048 rows of 5120 x 5120 float32, rank 32 on 2
// adapters 73, 75 and 75; 2047 rows of 17408 x 5120 bfloat16, rank 32 on 6 adapters 66 with each.
inline int outer_parts(int M, int D, int E, int R) {
  const int64_t tiles = outer_tiles(D, E, R), slots = 768;
  int best = 1;
  double least = 1e30;
  for (int p = 1; p <= kParts && (p == 1 || M / p >= 256); ++p) {
    const int rows = outer_part_rows(std::max(M, 1), p), n = (M + rows - 1) / std::max(rows, 1);
    if (p > 1 && n != p) continue;           // no empty part
    const double idle = (double)((tiles * p + slots - 1) / slots * slots) / (double)(tiles * p);
    const double cost = idle * M * 2.0 * D + (p > 1 ? p * 8.0 * E * R * D : 0.0) + 28672.0 * (double)(tiles * p);
    if (cost < least) least = cost, best = p;
  }
  return best;
}

// Whether a workgroup has one wave instead of four: where workgroups with little to sum (their fixed part counts then) are more
// than a round of 768, as four times as many of one wave do.  da and db at 5120 x 5120 in float32 on 16 adapters in 32 runs, rank 16:
// 128 rows 23 us with one and 34 with four, 256 rows 29 and 38 (all rows on one adapter: 28 and 30), 1024 rows on one adapter 78
// and 51; at 512 x 512, 256 rows 17 and 14.
inline bool outer_one_wave(int wgs, int rows, int E) {
  return wgs > 768 && rows <= std::max(kRows, 16 * std::min(E, 16));
}

OuterSum outer_sum(const OuterJob& j, int M, int E, int R) {
  const int parts = outer_parts(M, j.D, E, R);
  return {j.t, reinterpret_cast<const uint8_t*>(j.v), parts > 1 ? j.parts : j.g, (int)(outer_tiles(j.D, E, R) * parts), j.D,
          parts, outer_part_rows(std::max(M, 1), parts), j.rcontig};
}

template <int VT, int NR, int WAVES>
hipError_t go_waves(int M, int E, int R, const OuterSum& a, const OuterSum& b, const int32_t* ids, hipStream_t st) {
  if (!raise_lds_limit<lora_outer_kernel<VT, NR, WAVES>>()) return hipErrorInvalidValue;
  const int total = a.wgs + b.wgs;
  hipLaunchKernelGGL((lora_outer_kernel<VT, NR, WAVES>), dim3((unsigned)std::min(total, 1 << 20)), dim3(64 * WAVES),
                     (outer_lds<VT, NR, WAVES>()), st, M, E, R, total, a, b, ids);
  return hipGetLastError();
}
// The choice is each sum's own, so that its order of additions does not depend on the other's being computed.
template <int VT, int NR>
hipError_t go(int M, int E, int R, const OuterSum& a, const OuterSum& b, const int32_t* ids, hipStream_t st) {
  const bool one = outer_one_wave(a.wgs, a.part_rows, E);
  if (b.wgs > 0 && outer_one_wave(b.wgs, b.part_rows, E) != one) {
    OuterSum none = b;
    none.wgs = 0;
    const hipError_t err = go<VT, NR>(M, E, R, a, none, ids, st);
    return err != hipSuccess ? err : go<VT, NR>(M, E, R, b, none, ids, st);
  }
  if (one) return go_waves<VT, NR, 1>(M, E, R, a, b, ids, st);
  return go_waves<VT, NR, 4>(M, E, R, a, b, ids, st);
}
template <int VT, typename... A>
hipError_t by_rank(int M, int E, int R, const A&... a) {
  if (R <= 16) return go<VT, 1>(M, E, R, a...);
  if (R <= 32) return go<VT, 2>(M, E, R, a...);
  return go<VT, 4>(M, E, R, a...);
}
template <typename... A>
hipError_t by_type(XType vt, const A&... a) {
  if (vt == X_F32) return by_rank<X_F32>(a...);
  if (vt == X_BF16) return by_rank<X_BF16>(a...);
  return by_rank<X_F16>(a...);
}

}  // namespace

size_t lora_outer_bytes(int M, int D, int E, int R) {
  const int parts = outer_parts(M, D, E, R);
  return parts > 1 ? (size_t)parts * E * R * D * 4 : 0;
}

hipError_t lora_outer(int M, int E, int R, const OuterJob* jobs, int count, const int32_t* ids, hipStream_t st) {
  const OuterSum none{nullptr, nullptr, nullptr, 0, 0, 1, kRows, false};
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i) tiles += outer_tiles(jobs[i].D, E, R);
  if (tiles > (1 << 27)) return hipErrorInvalidValue;     // gradients beyond any memory; workgroups (up to 8 a tile) are counted in int
  return by_type(jobs[0].vt, M, E, R, outer_sum(jobs[0], M, E, R), count > 1 ? outer_sum(jobs[1], M, E, R) : none, ids, st);
}

hipError_t lora_outer_join(int M, int E, int R, const OuterJob* jobs, int count, hipStream_t st) {
  JoinSum join[2] = {{nullptr, nullptr, 0, 1}, {nullptr, nullptr, 0, 1}};
  for (int i = 0; i < count; ++i) {
    const int parts = outer_parts(M, jobs[i].D, E, R);
    if (parts > 1)
      join[i] = {reinterpret_cast<const f32x4*>(jobs[i].parts), reinterpret_cast<f32x4*>(jobs[i].g),
                 (int64_t)E * R * jobs[i].D / 4, parts};
  }
  const int64_t n4 = join[0].n4 + join[1].n4;
  if (n4 == 0) return hipSuccess;
  hipLaunchKernelGGL(lora_join_kernel, dim3((unsigned)std::min<int64_t>((n4 + 255) / 256, 2048)), dim3(256), 0, st, join[0],
                     join[1]);
  return hipGetLastError();
}

}  // namespace wq
