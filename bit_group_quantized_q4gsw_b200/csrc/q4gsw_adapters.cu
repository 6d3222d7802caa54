// q4gsw_adapters.cu - the low-rank half of a projection with an adapter for
// every token, and the gradients of the adapters (sm_100a).
//
// Three kernels over the tiles of a plan (16 tokens of one adapter each):
//   down   u = x A^T (forward), v = s d_y B (backward): the intermediate, fp32 [M][r]
//   up     the low-rank term s u B^T (or v A) with the residual, fp16 [M][C], left in
//          the output's place: the base product then adds itself as to any residual
//   grad   d_A = v^T x, d_B = s d_y^T u over the tokens of each adapter, fp32
// so that the base product runs on its own routes unchanged, at any number of
// tokens and with either kind of scales.
//
// The intermediate stays in fp32: rounded to fp16 it would put 2^-11 of error into
// fp32 gradients, and small gradients would fall below fp16's range.  `up` takes it
// to the tensor cores as two fp16 parts of each row divided by a power of two near
// the row's largest value (2^-24 of that), `grad` as two tf32 parts (2^-22 of each
// value), in which fp16 activations are exact.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdio>

#include "q4gsw_adapters.cuh"
#include "q4gsw_common.cuh"
#include "q4gsw_internal.h"

namespace cg = cooperative_groups;

namespace q4gsw {
namespace ma {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// Coherent loads: the operands come from kernels that may have run on this SM while
// this grid was already launched (programmatic dependent launch), and only the
// coherent path is documented to see their writes behind griddepcontrol.wait.
__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_v2(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_u32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_u16(const void* p) {
  unsigned short v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ int ld_int(const int32_t* p) { return (int)ld_u32(p); }
__device__ __forceinline__ float ld_f32(const float* p) { return __uint_as_float(ld_u32(p)); }

// BYTES bytes (a multiple of 2) at p, aligned to the largest power of two that
// divides BYTES, up to 16: into BYTES / 4 words, the last one half filled where
// BYTES is an odd number of halves.
template <int BYTES>
__device__ __forceinline__ void load_bytes(uint32_t (&w)[(BYTES + 3) / 4], const void* p) {
  const char* c = static_cast<const char*>(p);
  if constexpr (BYTES % 16 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = ld_v4(c + 16 * i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else if constexpr (BYTES % 8 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 8; ++i) {
      const uint2 v = ld_v2(c + 8 * i);
      w[2 * i] = v.x;
      w[2 * i + 1] = v.y;
    }
  } else if constexpr (BYTES % 4 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) w[i] = ld_u32(c + 4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 2; ++i) {
      const uint32_t v = ld_u16(c + 2 * i);
      w[i / 2] = i % 2 ? w[i / 2] | v << 16 : v;
    }
  }
}

// halves i of two registers: (lo.half[i], hi.half[i])
__device__ __forceinline__ uint32_t pair_halves(uint32_t lo, uint32_t hi, int i) {
  return prmt(lo, hi, i ? 0x7632u : 0x5410u);
}

// ---------------------------------------------------------------- down
// acc += the products of chunks [s_begin, s_end) of 64 columns of the rows a0 (g) and
// a1 (g + 8) of a tile with an adapter's matrix: P(c, j) = mat[j][c] when BY_ROWS
// (A [r, K]), mat[c][j] else (B [N, r]); r = 8 RJ.  Column n of tensor-core tile j is
// rank 8 j + n by rows, RJ n + j else (a lane then reads RJ ranks of a row at once).
//
// Lane t of a quad has columns c0 .. c0 + 15, c0 = 64 ch + 16 t, of both operands, and
// step s of the four takes (c0 + 2 s, + 1) as contraction indices 2 t, 2 t + 1 and
// (c0 + 8 + 2 s, + 1) as 2 t + 8, 2 t + 9.
//
// U chunks' loads are issued together: a warp with few chunks has one round of latency.
template <bool BY_ROWS, int RJ, int U>
__device__ __forceinline__ void down_chunks(const __half* mat, const __half* a0, const __half* a1, int C, int s_begin,
                                            int s_end, int g, int t, float (&acc)[RJ][4]) {
  constexpr int R = 8 * RJ;
  constexpr int PW = BY_ROWS ? 8 : (RJ + 1) / 2;      // words of the matrix per row of fragments
  const uint4 z4 = make_uint4(0u, 0u, 0u, 0u);
  for (int first = s_begin; first < s_end; first += U) {
    uint4 xv[U][4];
    uint32_t p[U][BY_ROWS ? RJ : 16][PW];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c0 = 64 * (first + u) + 16 * t;
      const bool live = first + u < s_end;
      const bool in0 = live && c0 + 8 <= C, in1 = live && c0 + 16 <= C;   // C % 8 == 0: 8 columns are in or out
      xv[u][0] = in0 ? ld_v4(a0 + c0) : z4;
      xv[u][1] = in1 ? ld_v4(a0 + c0 + 8) : z4;
      xv[u][2] = in0 ? ld_v4(a1 + c0) : z4;
      xv[u][3] = in1 ? ld_v4(a1 + c0 + 8) : z4;
      if constexpr (BY_ROWS) {
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          const __half* row = mat + (size_t)(8 * j + g) * C + c0;
          const uint4 q0 = in0 ? ld_v4(row) : z4, q1 = in1 ? ld_v4(row + 8) : z4;
          p[u][j][0] = q0.x, p[u][j][1] = q0.y, p[u][j][2] = q0.z, p[u][j][3] = q0.w;
          p[u][j][4] = q1.x, p[u][j][5] = q1.y, p[u][j][6] = q1.z, p[u][j][7] = q1.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
#pragma unroll
          for (int q = 0; q < PW; ++q) p[u][e][q] = 0u;
          if (e < 8 ? in0 : in1) load_bytes<2 * RJ>(p[u][e], mat + (size_t)(c0 + e) * R + RJ * g);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t* x0 = reinterpret_cast<const uint32_t*>(&xv[u][0]);
      const uint32_t* x1 = reinterpret_cast<const uint32_t*>(&xv[u][2]);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t af[4] = {x0[s], x1[s], x0[4 + s], x1[4 + s]};
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          uint32_t bf[2];
          if constexpr (BY_ROWS) {
            bf[0] = p[u][j][s];
            bf[1] = p[u][j][4 + s];
          } else {
            bf[0] = pair_halves(p[u][2 * s][j / 2], p[u][2 * s + 1][j / 2], j % 2);
            bf[1] = pair_halves(p[u][8 + 2 * s][j / 2], p[u][9 + 2 * s][j / 2], j % 2);
          }
          mma_16816(acc[j], af, bf);
        }
      }
    }
  }
}
// the sums as [row][rank]: D has rows g, g + 8 and columns 2 t, 2 t + 1 of tile j
template <bool BY_ROWS, int RJ>
__device__ __forceinline__ void down_park(const float (&acc)[RJ][4], float (*red)[8 * RJ], int g, int t) {
#pragma unroll
  for (int j = 0; j < RJ; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int col = 2 * t + (q & 1);
      red[g + 8 * (q >> 1)][BY_ROWS ? 8 * j + col : RJ * col + j] = acc[j][q];
    }
}

// out[m][j] = f sum_c act[m][c] P(c, j) for the tokens m of a tile, P and f (where scale
// is given) of the tile's adapter.
//
// A CTA has WT consecutive tiles, eight warps 8 / WT to a tile; the warps of a tile and
// the KS CTAs of the cluster (grid = (slots / WT, KS)) split the contraction.  The
// warps' sums are added in shared memory and the CTAs' through distributed shared
// memory, both in a fixed order.  mma.sync m16n8k16: the work is bound by bytes (the
// activations once, the adapter's matrix once a CTA, from L1 by the warps of its other
// tiles) and by the latency of the loads.
template <bool BY_ROWS, int RJ, int WT>
__global__ void __launch_bounds__(kThreads)
q4gsw_adapters_down_kernel(const __half* act, const __half* proj, const float* scale, const int32_t* plan, float* out,
                           int M, int L, int C) {
  constexpr int R = 8 * RJ, WK = kWarps / WT;
  __shared__ float red[kWarps][kTileRows][R];
  __shared__ float recv[WT][kTileRows][R];     // [sender][owned row] of each tile
  griddep_wait();
  griddep_launch_dependents();     // behind the wait: what ran before has been written when the next kernel starts
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  const int KS = gridDim.y, ks = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int slots = plan_slots(M, L), slot0 = blockIdx.x * WT;
  const int slot = slot0 + warp / WK;
  const int adapter = slot < slots ? ld_int(P.tile + slot) : kNoTile;
  const int32_t* rows = P.rows + (size_t)slot * kTileRows;
  // tiles in use come first: where the first is unused, so is the whole cluster
  if (WT == 1 ? adapter == kNoTile : ld_int(P.tile + slot0) == kNoTile) return;
  if (KS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  float acc[RJ][4];
#pragma unroll
  for (int j = 0; j < RJ; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[j][q] = 0.f;
  if (adapter >= 0) {
    const __half* mat = proj + (size_t)adapter * R * C;
    // rows that the tile lacks read its first (never stored)
    const int ra = ld_int(rows + g), rb = ld_int(rows + g + 8), r0 = ld_int(rows);
    const __half* a0 = act + (size_t)(ra < 0 ? r0 : ra) * C;
    const __half* a1 = act + (size_t)(rb < 0 ? r0 : rb) * C;
    const int chunks = (C + 63) / 64;   // C % 8 == 0: a group of 8 columns is wholly in or out
    const int parts = KS * WK, part = ks * WK + warp % WK;
    const int s_begin = (int)((long long)part * chunks / parts), s_end = (int)((long long)(part + 1) * chunks / parts);
    down_chunks<BY_ROWS, RJ, (RJ <= 2 ? 2 : 1)>(mat, a0, a1, C, s_begin, s_end, g, t, acc);
  }
  down_park<BY_ROWS, RJ>(acc, red[warp], g, t);
  __syncthreads();
  // the sums of row `row` of tile `tile` over its warps; a tile without an adapter has zeros
  auto own = [&](int tile, int row, int j) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) s += red[tile * WK + w][row][j];
    return s;
  };
  const int owned = kTileRows / KS;      // rows of each tile that this CTA writes (KS is a power of two)
  if (KS > 1) {
    // every CTA of the cluster has started (arrived above): remote stores are safe
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    for (int e = threadIdx.x; e < WT * kTileRows * R; e += kThreads) {
      const int tile = e / (kTileRows * R), row = e / R % kTileRows, j = e % R;
      *cluster.map_shared_rank(&recv[tile][ks * owned + row % owned][j], row / owned) = own(tile, row, j);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  for (int e = threadIdx.x; e < WT * owned * R; e += kThreads) {
    const int tile = e / (owned * R), row = e / R % owned, j = e % R;
    if (slot0 + tile >= slots) break;
    const int m = ld_int(P.rows + (size_t)(slot0 + tile) * kTileRows + ks * owned + row);
    if (m < 0) continue;
    const int a = ld_int(P.tile + slot0 + tile);
    float s = 0.f;
    if (KS > 1) {
      for (int q = 0; q < KS; ++q) s += recv[tile][q * owned + row][j];
    } else {
      s = own(tile, row, j);
    }
    out[(size_t)m * R + j] = a >= 0 && scale ? ld_f32(scale + a) * s : s;
  }
}

// ---------------------------------------------------------------- up
// out[m][c] = fp16(res[m][c] + f sum_j q[m][j] P(c, j)): P(c, j) = proj[c][j] when
// BY_ROWS (B [N, r]), proj[j][c] else (A [r, K]).  Tokens without an adapter get
// their residual, or zeros.
//
// A warp has one tile's 16 tokens and blocks of 64 columns.  Column 8 s(n) + i of a
// block, s(2 t) = t and s(2 t + 1) = 4 + t, is column n of tensor-core tile i, so that a
// lane's results are columns of its two rows in two vectors of 16 bytes, which the
// four lanes of a quad read (the residual, by columns also the matrix) and write side by
// side, and nothing goes through shared memory.

// The intermediate's fragments: a lane has 2 RJ ranks in parts of PART, the parts of
// the four lanes of a quad side by side (whole sectors); its ranks e = 4 s .. 4 s + 3 are
// the indices 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of step s.  Two fp16 parts, hi and lo, of the
// row over 2^k, k the exponent of its largest value.
template <int RJ>
struct UpTile {
  static constexpr int KT = (RJ + 1) / 2;    // tensor-core steps of 16 ranks
  static constexpr int PART = RJ % 4 == 0 ? 8 : RJ % 2 == 0 ? 4 : 2;     // ranks
  static constexpr int PARTS = 2 * RJ / PART;
  uint32_t hi[KT][4], lo[KT][4];
  float back[2];      // f 2^k of rows g and g + 8
  __device__ __forceinline__ static int rank_of(int e, int t) { return 4 * PART * (e / PART) + PART * t + e % PART; }
  // `load(h, e, v0, v1)`: ranks rank_of(e), + 1 (e even) of row g + 8 h
  template <class F>
  __device__ __forceinline__ void fill(float f, F&& load) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[4 * KT];
#pragma unroll
      for (int e = 0; e < 4 * KT; ++e) v[e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * RJ; e += 2) load(h, e, v[e], v[e + 1]);
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 4 * KT; ++e) top = fmaxf(top, fabsf(v[e]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^k and 2^-k from the exponent bits, k kept where both are normal numbers;
      // an infinite or NaN value stays what it is
      int k = (int)(__float_as_uint(top) >> 23) - 127;
      k = max(-126, min(k, 126));
      const float down = __uint_as_float((uint32_t)(127 - k) << 23);
      back[h] = f * __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
      for (int s = 0; s < KT; ++s)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float w0 = v[4 * s + 2 * q] * down, w1 = v[4 * s + 2 * q + 1] * down;
          const __half2 p = __floats2half2_rn(w0, w1);
          const float2 pf = __half22float2(p);
          hi[s][2 * q + h] = h2_as_u32(p);
          // (an infinity leaves no rest)
          lo[s][2 * q + h] = h2_as_u32(__floats2half2_rn(isinf(w0) ? 0.f : w0 - pf.x, isinf(w1) ? 0.f : w1 - pf.y));
        }
    }
  }
};

// One block of 64 columns from `base` on, of tokens m[0] (row g) and m[1] (row g + 8).
template <bool BY_ROWS, int RJ>
__device__ __forceinline__ void up_block(const __half* mat, const UpTile<RJ>& q, bool adapted, const int (&m)[2],
                                         int base, int C, const __half* res, __half* out, int g, int t) {
  using T = UpTile<RJ>;
  constexpr int R = 8 * RJ, KT = T::KT, PART = T::PART;
  const int sg = (g >> 1) + 4 * (g & 1);
  float acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  if (adapted) {
    const bool in = base + 8 * sg < C;     // C % 8 == 0
    if constexpr (BY_ROWS) {
      uint32_t w[8][RJ];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int p = 0; p < T::PARTS; ++p) {
          uint32_t part[PART / 2];
#pragma unroll
          for (int e = 0; e < PART / 2; ++e) part[e] = 0u;
          if (in) load_bytes<2 * PART>(part, mat + (size_t)(base + 8 * sg + i) * R + T::rank_of(p * PART, t));
#pragma unroll
          for (int e = 0; e < PART / 2; ++e) w[i][p * (PART / 2) + e] = part[e];
        }
      }
#pragma unroll
      for (int s = 0; s < KT; ++s)
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t bf[2] = {w[i][2 * s], 2 * s + 1 < RJ ? w[i][2 * s + 1 < RJ ? 2 * s + 1 : 0] : 0u};
            mma_16816(acc[i], part ? q.hi[s] : q.lo[s], bf);
          }
    } else {
#pragma unroll
      for (int s = 0; s < KT; ++s) {
        uint4 w[4];     // ranks 4 s .. 4 s + 3 of the lane, 8 columns each
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = in && 4 * s + e < 2 * RJ ? ld_v4(mat + (size_t)T::rank_of(4 * s + e, t) * C + base + 8 * sg)
                                          : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&w[0]);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&w[1]);
        const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&w[2]);
        const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&w[3]);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t bf[2] = {pair_halves(w0[i / 2], w1[i / 2], i % 2), pair_halves(w2[i / 2], w3[i / 2], i % 2)};
            mma_16816(acc[i], part ? q.hi[s] : q.lo[s], bf);
          }
      }
    }
  }
  // columns base + 8 t + i (acc[i][0], row g; [2], row g + 8) and + 32 + i ([1], [3])
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (m[h] < 0) continue;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = base + 8 * t + 32 * e;
      if (c >= C) continue;
      const size_t at = (size_t)m[h] * C + c;
      uint4 r = make_uint4(0u, 0u, 0u, 0u);
      if (res) r = *reinterpret_cast<const uint4*>(res + at);
      const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 rf = __half22float2(u32_as_h2(rw[i]));
        o[i] = !adapted ? rw[i]
                        : h2_as_u32(__floats2half2_rn(fmaf(q.back[h], acc[2 * i][2 * h + e], rf.x),
                                                      fmaf(q.back[h], acc[2 * i + 1][2 * h + e], rf.y)));
      }
      *reinterpret_cast<uint4*>(out + at) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <bool BY_ROWS, int RJ>
__global__ void __launch_bounds__(kThreads)
q4gsw_adapters_up_kernel(const float* inter, const __half* proj, const float* scale, const int32_t* plan,
                         const __half* res, __half* out, int M, int L, int C, int tile_warps, int blocks_per_warp) {
  constexpr int R = 8 * RJ;
  griddep_launch_dependents();
  griddep_wait();
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int slot = blockIdx.x * tile_warps + warp % tile_warps;
  if (slot >= plan_slots(M, L)) return;
  const int adapter = ld_int(P.tile + slot);
  if (adapter == kNoTile) return;
  const int blocks = (C + 63) / 64;
  const int first = (blockIdx.y * (kWarps / tile_warps) + warp / tile_warps) * blocks_per_warp;
  const int last = min(first + blocks_per_warp, blocks);
  const int32_t* rows = P.rows + (size_t)slot * kTileRows;
  const int m[2] = {ld_int(rows + g), ld_int(rows + g + 8)};
  UpTile<RJ> q;
  q.fill(adapter >= 0 && scale ? ld_f32(scale + adapter) : 1.f, [&](int h, int e, float& v0, float& v1) {
    if (m[h] < 0 || adapter < 0) return;
    const uint2 w = ld_v2(inter + (size_t)m[h] * R + UpTile<RJ>::rank_of(e, t));
    v0 = __uint_as_float(w.x);
    v1 = __uint_as_float(w.y);
  });
  const __half* mat = proj + (size_t)(adapter < 0 ? 0 : adapter) * R * C;
  for (int b = first; b < last; ++b)
    up_block<BY_ROWS, RJ>(mat, q, adapter >= 0, m, 64 * b, C, res, out, g, t);
}

// ---------------------------------------------------------------- down and up in one
// For few tiles: a cluster of KS CTAs has one tile.  Its CTAs split the contraction of
// `down`, each gets the sums of all of them (every CTA writes its own to every other's
// shared memory, added in rank order), and they split the columns of `up`.  One launch
// and one exchange in place of two launches and a trip through memory; `inter` is
// written for the backward pass.  FWD: x, A, B; else d_y, B, A.
template <bool FWD, int RJ, int U>
__global__ void __launch_bounds__(kThreads, U == 1 && RJ <= 2 ? 3 : 1)
q4gsw_adapters_low_kernel(const __half* act, const __half* mat_down, const __half* mat_up, const float* scale,
                          const int32_t* plan, float* inter, const __half* res, __half* out, int M, int L, int C_down,
                          int C_up) {
  constexpr int R = 8 * RJ;
  extern __shared__ __align__(16) float low_smem[];
  auto red = reinterpret_cast<float (*)[kTileRows][R]>(low_smem);                       // [kWarps]
  auto recv = reinterpret_cast<float (*)[kTileRows][R]>(low_smem + kWarps * kTileRows * R);   // [KS], by sender
  griddep_wait();
  griddep_launch_dependents();     // behind the wait: what ran before has been written when the next kernel starts
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  const int KS = gridDim.y, ks = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int adapter = ld_int(P.tile + blockIdx.x);
  if (adapter == kNoTile) return;
  const int32_t* rows = P.rows + (size_t)blockIdx.x * kTileRows;
  const int m[2] = {ld_int(rows + g), ld_int(rows + g + 8)};
  UpTile<RJ> q;
  const __half* up = mat_up + (size_t)(adapter < 0 ? 0 : adapter) * R * C_up;
  const int blocks = (C_up + 63) / 64;
  if (adapter >= 0) {
    if (KS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    // the first block's part of `up`'s matrix on its way to L2 meanwhile
    const int b0 = ks * kWarps + warp;
    if (b0 < blocks) {
      const int cols = min(64, C_up - 64 * b0);
      if (FWD) {
        for (int e = lane; e < cols * R / 64; e += 32) prefetch_l2(up + (size_t)(64 * b0) * R + 64 * e);
      } else {
        for (int e = lane; e < R; e += 32) prefetch_l2(up + (size_t)e * C_up + 64 * b0);
      }
    }
    const int r0 = ld_int(rows);
    const __half* a0 = act + (size_t)(m[0] < 0 ? r0 : m[0]) * C_down;
    const __half* a1 = act + (size_t)(m[1] < 0 ? r0 : m[1]) * C_down;
    const int chunks = (C_down + 63) / 64, parts = KS * kWarps, part = ks * kWarps + warp;
    const int s_begin = (int)((long long)part * chunks / parts), s_end = (int)((long long)(part + 1) * chunks / parts);
    float acc[RJ][4];
#pragma unroll
    for (int j = 0; j < RJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    down_chunks<FWD, RJ, U>(mat_down + (size_t)adapter * R * C_down, a0, a1, C_down, s_begin, s_end, g, t, acc);
    down_park<FWD, RJ>(acc, red[warp], g, t);
    __syncthreads();
    if (KS > 1) {
      // every CTA of the cluster has started (arrived above): remote stores are safe
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      cg::cluster_group cluster = cg::this_cluster();
      for (int e = threadIdx.x; e < kTileRows * R; e += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += red[w][e / R][e % R];
        for (int k = 0; k < KS; ++k) *cluster.map_shared_rank(&recv[ks][e / R][e % R], k) = s;
      }
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    const float f = scale ? ld_f32(scale + adapter) : 1.f;
    for (int e = threadIdx.x; e < kTileRows * R; e += kThreads) {
      float s = 0.f;
      if (KS > 1) {
        for (int k = 0; k < KS; ++k) s += recv[k][e / R][e % R];
      } else {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += red[w][e / R][e % R];
      }
      if (!FWD) s *= f;
      red[0][e / R][e % R] = s;      // (each element is read and written by one thread)
      const int to = ld_int(rows + e / R);
      if (ks == 0 && to >= 0) inter[(size_t)to * R + e % R] = s;
    }
    __syncthreads();
    q.fill(FWD ? f : 1.f, [&](int h, int e, float& v0, float& v1) {
      const float* v = &red[0][g + 8 * h][UpTile<RJ>::rank_of(e, t)];
      v0 = v[0];
      v1 = v[1];
    });
  } else if (ks == 0) {
    for (int e = threadIdx.x; e < kTileRows * R; e += kThreads) {
      const int to = ld_int(rows + e / R);
      if (to >= 0) inter[(size_t)to * R + e % R] = 0.f;
    }
  }
  for (int b = ks * kWarps + warp; b < blocks; b += KS * kWarps)
    up_block<FWD, RJ>(up, q, adapter >= 0, m, 64 * b, C_up, res, out, g, t);
}

// ---------------------------------------------------------------- grad
// G_a(c, j) = f sum over the tokens m of adapter a of act[m][c] q[m][j], fp32, as
// rows [c][r] (BY_ROWS: d_B [N, r]) or [r][c] (d_A [r, K]).  f the adapter's factor
// (scale given) or 1.
//
// mma.sync m16n8k8 tf32, 16 ranks x 8 columns x 8 tokens: the activations are exact
// in tf32, q goes in as two parts.  Column CW / 8 n + i of a block of CW columns is
// column n of tensor-core tile i, so that a lane reads its columns of a token's row
// as one vector, straight into the fragments.  A CTA has one block of columns of one
// adapter; its warps take the tokens eight at a time in turn and their sums are added
// in shared memory in a fixed order.
__device__ __forceinline__ uint32_t to_tf32(float v) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void mma_1688_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int RJ>
struct GradTile {
  static constexpr int MT = (RJ + 1) / 2;          // tensor-core tiles of 16 ranks
  static constexpr int CW = MT <= 2 ? 64 : 32;     // columns of a warp: at most 64 sums a lane
  static constexpr int V = CW / 8;                 // columns of a lane
};

// One of the two gradients: the columns' activations and the other factor.
struct GradSide {
  const __half* act;
  const float* q;
  const float* scale;
  float* out;
  int C;
};

// The CTA's sums in shared memory: rows of the output, padded by four values.
template <int RJ, int TS>
__host__ __device__ constexpr int grad_tile_floats() {
  constexpr int W = kWarps / TS * GradTile<RJ>::CW, R = 8 * RJ;
  return (W * (R + 4)) > (R * (W + 4)) ? W * (R + 4) : R * (W + 4);
}

template <bool BY_ROWS, int RJ, int TS>
__device__ __forceinline__ void grad_block(const GradSide& a, const PlanView& P, int group, int accumulate, float* tile) {
  using T = GradTile<RJ>;
  constexpr int R = 8 * RJ, MT = T::MT, CW = T::CW, V = T::V;
  constexpr int CB = kWarps / TS;              // blocks of columns of the CTA
  constexpr int W = CB * CW;
  constexpr int PITCH = (BY_ROWS ? R : W) + 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int adapter = blockIdx.y;
  const int base = W * group;
  const int begin = ld_int(P.first + adapter), end = ld_int(P.first + adapter + 1);
  float* dst = a.out + (size_t)adapter * R * a.C;
  const int split = warp / CB, block = warp % CB;
  if (begin < end) {
    float acc[MT][V][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[m][i][k] = 0.f;
    const int col = base + CW * block + V * g;
    const bool in = col < a.C;        // C % 8 == 0, V is 4 or 8
    // tokens of a step: rows t and t + 4 of this lane; the next step's are loaded
    // before this one's products
    float w[MT][4];
    uint32_t x[2][V / 2];
    int token[2];
    auto index = [&](int p0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) token[h] = p0 + t + 4 * h < end ? ld_int(P.order + p0 + t + 4 * h) : -1;
    };
    auto load = [&] {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = token[h];
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int j = 16 * b + g + 8 * k;
            w[b][2 * h + k] = m >= 0 && j < R ? ld_f32(a.q + (size_t)m * R + j) : 0.f;
          }
        if (m >= 0 && in) {
          load_bytes<2 * V>(x[h], a.act + (size_t)m * a.C + col);
        } else {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) x[h][i] = 0u;
        }
      }
    };
    const int p_first = begin + 8 * split;
    index(p_first);
    load();
    index(p_first + 8 * TS);
    for (int p0 = p_first; p0 < end; p0 += 8 * TS) {
      uint32_t hi[MT][4], lo[MT][4], now[2][V / 2];
#pragma unroll
      for (int b = 0; b < MT; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hi[b][k] = to_tf32(w[b][k]);
          lo[b][k] = to_tf32(w[b][k] - __uint_as_float(hi[b][k]));
        }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < V / 2; ++i) now[h][i] = x[h][i];
      load();      // the next step's (nothing past the end)
      index(p0 + 16 * TS);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 f0 = __half22float2(u32_as_h2(now[0][i / 2])), f1 = __half22float2(u32_as_h2(now[1][i / 2]));
          const uint32_t b0 = __float_as_uint(i % 2 ? f0.y : f0.x), b1 = __float_as_uint(i % 2 ? f1.y : f1.x);
#pragma unroll
          for (int b = 0; b < MT; ++b) mma_1688_tf32(acc[b][i], part ? hi[b] : lo[b], b0, b1);
        }
    }
    // the splits' sums into the tile, one after another
#pragma unroll 1
    for (int s = 0; s < TS; ++s) {
      if (split == s) {
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
          for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = 16 * b + g + 8 * (k >> 1), c = CW * block + V * (2 * t + (k & 1)) + i;
              if (j >= R) continue;
              float* at = tile + (BY_ROWS ? c * PITCH + j : j * PITCH + c);
              *at = s ? *at + acc[b][i][k] : acc[b][i][k];
            }
      }
      __syncthreads();
    }
  } else if (accumulate) {
    return;
  }
  const float f = a.scale ? ld_f32(a.scale + adapter) : 1.f;
  // rows of the output, four values a thread
  for (int e = threadIdx.x; e < W * R / 4; e += kThreads) {
    const int row = BY_ROWS ? e / (R / 4) : e / (W / 4), x4 = BY_ROWS ? e % (R / 4) : e % (W / 4);
    if ((BY_ROWS ? base + row : base + 4 * x4) >= a.C) continue;
    float4* at = reinterpret_cast<float4*>(BY_ROWS ? dst + (size_t)(base + row) * R + 4 * x4
                                                   : dst + (size_t)row * a.C + base + 4 * x4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (begin < end) {
      v = *reinterpret_cast<const float4*>(tile + row * PITCH + 4 * x4);
      v = make_float4(f * v.x, f * v.y, f * v.z, f * v.w);
      if (accumulate) {
        const float4 o = *at;
        v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
      }
    }
    *at = v;
  }
}

template <int RJ, int TS>
__global__ void __launch_bounds__(kThreads)
q4gsw_adapters_grad_kernel(const GradSide da, const GradSide db, const int32_t* plan, int M, int L, int groups_a,
                           int accumulate) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ __align__(16) float tile[grad_tile_floats<RJ, TS>()];
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  if ((int)blockIdx.x < groups_a) grad_block<false, RJ, TS>(da, P, blockIdx.x, accumulate, tile);
  else grad_block<true, RJ, TS>(db, P, blockIdx.x - groups_a, accumulate, tile);
}

// The rank as a compile-time constant.
#define Q4_RANKS(RJ_, CALL) \
  switch (RJ_) {            \
    case 1: CALL(1);        \
    case 2: CALL(2);        \
    case 3: CALL(3);        \
    case 4: CALL(4);        \
    case 5: CALL(5);        \
    case 6: CALL(6);        \
    case 7: CALL(7);        \
    default: CALL(8);       \
  }

}  // namespace ma

static void serialize(cudaLaunchAttribute& a) {
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
}

template <bool BY_ROWS, int RJ>
static cudaError_t down_tiles(cudaLaunchConfig_t& cfg, int wt, const __half* a, const __half* p, const float* scale,
                              const AdaptersRef& ad, float* out, int M, int C) {
  return wt == 1 ? cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_down_kernel<BY_ROWS, RJ, 1>, a, p, scale, ad.plan, out,
                                      M, ad.L, C)
                 : cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_down_kernel<BY_ROWS, RJ, 4>, a, p, scale, ad.plan, out,
                                      M, ad.L, C);
}

cudaError_t launch_adapters_down(const AdaptersRef& ad, const uint16_t* act, bool by_rows, const uint16_t* proj,
                                 const float* scale, int M, int C, float* out, cudaStream_t stream) {
  const int slots = ma::plan_slots(M, ad.L), sms = sm_count(current_device());
  const int wt = slots >= 64 ? 4 : 1;
  const int groups = (slots + wt - 1) / wt;
  // contraction splits: about two CTAs per SM, a chunk of 64 columns per warp, clusters of at most 8
  const int chunks = (C + 63) / 64;
  int KS = 1;
  while (KS < 8 && groups * KS < 2 * sms && chunks / (2 * KS) >= ma::kWarps / wt) KS *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(groups, KS, 1);
  cfg.blockDim = dim3(ma::kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  serialize(attr[0]);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = KS;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const __half* a = reinterpret_cast<const __half*>(act);
  const __half* p = reinterpret_cast<const __half*>(proj);
#define Q4_DOWN(RJ_)                                                               \
  return by_rows ? down_tiles<true, RJ_>(cfg, wt, a, p, scale, ad, out, M, C)      \
                 : down_tiles<false, RJ_>(cfg, wt, a, p, scale, ad, out, M, C)
  Q4_RANKS(ad.r / 8, Q4_DOWN)
#undef Q4_DOWN
}

cudaError_t launch_adapters_up(const AdaptersRef& ad, const float* inter, bool by_rows, const uint16_t* proj,
                               const float* scale, int M, int C, const uint16_t* res, uint16_t* out,
                               cudaStream_t stream) {
  const int slots = ma::plan_slots(M, ad.L), sms = sm_count(current_device());
  int tile_warps = 1;
  while (tile_warps < ma::kWarps && tile_warps < slots) tile_warps *= 2;
  const int col_warps = ma::kWarps / tile_warps;
  const int blocks = (C + 63) / 64, groups = (slots + tile_warps - 1) / tile_warps;
  // blocks of columns of a warp, one after another: as many as leave four CTAs per SM
  int per = (int)((long long)groups * blocks / col_warps / (4 * sms));
  per = per < 1 ? 1 : per > 16 ? 16 : per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(groups, (blocks + col_warps * per - 1) / (col_warps * per), 1);
  cfg.blockDim = dim3(ma::kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  serialize(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const __half* p = reinterpret_cast<const __half*>(proj);
  const __half* rs = reinterpret_cast<const __half*>(res);
  __half* o = reinterpret_cast<__half*>(out);
#define Q4_UP(RJ_)                                                                                                \
  return by_rows ? cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_up_kernel<true, RJ_>, inter, p, scale, ad.plan, rs, o, \
                                      M, ad.L, C, tile_warps, per)                                                \
                 : cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_up_kernel<false, RJ_>, inter, p, scale, ad.plan, rs, o, \
                                      M, ad.L, C, tile_warps, per)
  Q4_RANKS(ad.r / 8, Q4_UP)
#undef Q4_UP
}

template <bool FWD, int RJ, int U>
static cudaError_t low_form(cudaLaunchConfig_t& cfg, int KS, const __half* act, const __half* down, const __half* up,
                            const float* scale, const AdaptersRef& ad, float* inter, const __half* res, __half* out,
                            int M, int C_down, int C_up) {
  constexpr int kTile = (int)sizeof(float) * ma::kTileRows * 8 * RJ;
  auto kernel = ma::q4gsw_adapters_low_kernel<FWD, RJ, U>;
  static PerDeviceOnce once;
  const cudaError_t e = once_per_device(once, current_device(), [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (ma::kWarps + 8) * kTile);
  });
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = (ma::kWarps + (KS > 1 ? KS : 0)) * kTile;
  return cudaLaunchKernelEx(&cfg, kernel, act, down, up, scale, ad.plan, inter, res, out, M, ad.L, C_down, C_up);
}

bool adapters_low_fits(const AdaptersRef& ad, int M) {
  return ma::plan_slots(M, ad.L) <= 64;
}

cudaError_t launch_adapters_low(const AdaptersRef& ad, bool fwd, const uint16_t* act, const uint16_t* a,
                                const uint16_t* b, const float* scale, int M, int K, int N, float* inter,
                                const uint16_t* res, uint16_t* out, cudaStream_t stream) {
  const int slots = ma::plan_slots(M, ad.L);
  const int KS = 8;
  const bool deep = ((fwd ? K : N) + 63) / 64 > KS * ma::kWarps;      // more than a chunk a warp
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(slots, KS, 1);
  cfg.blockDim = dim3(ma::kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  serialize(attr[0]);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = KS;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const __half* x = reinterpret_cast<const __half*>(act);
  const __half* pa = reinterpret_cast<const __half*>(a);
  const __half* pb = reinterpret_cast<const __half*>(b);
  const __half* rs = reinterpret_cast<const __half*>(res);
  __half* o = reinterpret_cast<__half*>(out);
#define Q4_LOW(RJ_)                                                                                                   \
  {                                                                                                                   \
    constexpr int U = RJ_ <= 2 ? 4 : RJ_ <= 4 ? 2 : 1;                                                                \
    return fwd ? (deep ? low_form<true, RJ_, U>(cfg, KS, x, pa, pb, scale, ad, inter, rs, o, M, K, N)                 \
                       : low_form<true, RJ_, 1>(cfg, KS, x, pa, pb, scale, ad, inter, rs, o, M, K, N))                \
               : (deep ? low_form<false, RJ_, U>(cfg, KS, x, pb, pa, scale, ad, inter, rs, o, M, N, K)                \
                       : low_form<false, RJ_, 1>(cfg, KS, x, pb, pa, scale, ad, inter, rs, o, M, N, K));              \
  }
  Q4_RANKS(ad.r / 8, Q4_LOW)
#undef Q4_LOW
}

template <int RJ, int TS>
static cudaError_t grad_splits(cudaLaunchConfig_t& cfg, const AdaptersRef& ad, const ma::GradSide& da,
                               const ma::GradSide& db, int M, bool accumulate) {
  constexpr int W = ma::kWarps / TS * ma::GradTile<RJ>::CW;
  const int ga = (da.C + W - 1) / W, gb = (db.C + W - 1) / W;
  cfg.gridDim = dim3(ga + gb, ad.L, 1);
  return cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_grad_kernel<RJ, TS>, da, db, ad.plan, M, ad.L, ga, (int)accumulate);
}

cudaError_t launch_adapters_grad(const AdaptersRef& ad, const uint16_t* x, const float* v, float* d_a, int K,
                                 const uint16_t* d_y, const float* u, const float* scale, float* d_b, int N, int M,
                                 bool accumulate, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(ma::kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  serialize(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const ma::GradSide da{reinterpret_cast<const __half*>(x), v, nullptr, d_a, K};
  const ma::GradSide db{reinterpret_cast<const __half*>(d_y), u, scale, d_b, N};
  const int ts = M / ad.L >= 512 ? 8 : M / ad.L >= 128 ? 4 : 2;
#define Q4_GRAD(RJ_)                                                        \
  return ts == 8   ? grad_splits<RJ_, 8>(cfg, ad, da, db, M, accumulate)    \
         : ts == 4 ? grad_splits<RJ_, 4>(cfg, ad, da, db, M, accumulate)    \
                   : grad_splits<RJ_, 2>(cfg, ad, da, db, M, accumulate)
  Q4_RANKS(ad.r / 8, Q4_GRAD)
#undef Q4_GRAD
}

}  // namespace q4gsw
