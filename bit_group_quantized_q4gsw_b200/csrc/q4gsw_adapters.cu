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
// out[m][j] = f sum_c act[m][c] P(c, j) for the tokens m of a tile, P of the tile's
// adapter: P(c, j) = proj[j][c] when BY_ROWS (A [r, K]), proj[c][j] else (B [N, r]);
// f the adapter's factor (scale given) or 1.  r = 8 RJ.
//
// grid = (slots, KS), cluster (1, KS): the KS CTAs of a tile, and their eight warps,
// split the contraction; the warps' tiles are summed in shared memory and the CTAs'
// through distributed shared memory, both in a fixed order.  mma.sync m16n8k16: the
// work is bound by bytes (the activations once, the adapter's matrix once a tile)
// and, for few tokens, by the latency of its loads.
template <bool BY_ROWS, int RJ>
__global__ void __launch_bounds__(kThreads)
q4gsw_adapters_down_kernel(const __half* act, const __half* proj,
                           const float* scale, const int32_t* plan, float* out, int M, int L,
                           int C) {
  constexpr int R = 8 * RJ;
  __shared__ float red[kWarps][kTileRows][R];
  __shared__ float recv[8][8][R];     // [sender][owned row][rank], KS >= 2: at most 8 rows owned
  griddep_launch_dependents();
  griddep_wait();
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  const int KS = gridDim.y, ks = blockIdx.y;
  const int adapter = ld_int(P.tile + blockIdx.x);
  const int32_t* rows = P.rows + (size_t)blockIdx.x * kTileRows;
  if (adapter == kNoTile) return;
  if (adapter == kNoAdapter) {
    if (ks == 0)
      for (int e = threadIdx.x; e < kTileRows * R; e += kThreads) {
        const int m = ld_int(rows + e / R);
        if (m >= 0) out[(size_t)m * R + e % R] = 0.f;
      }
    return;
  }
  if (KS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const __half* mat = proj + (size_t)adapter * R * C;
  // rows that the tile lacks read its first (never stored)
  const int ra = ld_int(rows + g), rb = ld_int(rows + g + 8), r0 = ld_int(rows);
  const __half* a0 = act + (size_t)(ra < 0 ? r0 : ra) * C;
  const __half* a1 = act + (size_t)(rb < 0 ? r0 : rb) * C;
  const int chunks = (C + 63) / 64;   // C % 8 == 0: a group of 8 columns is wholly in or out
  const int c_begin = (int)((long long)ks * chunks / KS), c_end = (int)((long long)(ks + 1) * chunks / KS);
  const int s_begin = c_begin + warp * (c_end - c_begin) / kWarps;
  const int s_end = c_begin + (warp + 1) * (c_end - c_begin) / kWarps;
  float acc[RJ][4];
#pragma unroll
  for (int j = 0; j < RJ; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[j][q] = 0.f;
  const uint4 z4 = make_uint4(0u, 0u, 0u, 0u);
  // A chunk of 64 columns: lane t of a quad has columns c0 .. c0 + 15, c0 = 64 ch + 16 t,
  // of both operands, and step s of the four takes (c0 + 2 s, + 1) as contraction
  // indices 2 t, 2 t + 1 and (c0 + 8 + 2 s, + 1) as 2 t + 8, 2 t + 9.
#pragma unroll 2
  for (int ch = s_begin; ch < s_end; ++ch) {
    const int c0 = 64 * ch + 16 * t;
    const bool in0 = c0 + 8 <= C, in1 = c0 + 16 <= C;
    uint4 xv[4];
    xv[0] = in0 ? ld_v4(a0 + c0) : z4;
    xv[1] = in1 ? ld_v4(a0 + c0 + 8) : z4;
    xv[2] = in0 ? ld_v4(a1 + c0) : z4;
    xv[3] = in1 ? ld_v4(a1 + c0 + 8) : z4;
    const uint32_t* x0 = reinterpret_cast<const uint32_t*>(&xv[0]);
    const uint32_t* x1 = reinterpret_cast<const uint32_t*>(&xv[2]);
    if constexpr (BY_ROWS) {
      // rank 8 j + g is column g of tile j
      uint4 p[RJ][2];
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        const __half* row = mat + (size_t)(8 * j + g) * C + c0;
        p[j][0] = in0 ? ld_v4(row) : z4;
        p[j][1] = in1 ? ld_v4(row + 8) : z4;
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t af[4] = {x0[s], x1[s], x0[4 + s], x1[4 + s]};
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(p[j]);
          const uint32_t bf[2] = {w[s], w[4 + s]};
          mma_16816(acc[j], af, bf);
        }
      }
    } else {
      // rank RJ g + j is column g of tile j: a lane reads RJ ranks of a row at once
      uint32_t p[16][(RJ + 1) / 2];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e < 8 ? in0 : in1) {
          load_bytes<2 * RJ>(p[e], mat + (size_t)(c0 + e) * R + RJ * g);
        } else {
#pragma unroll
          for (int q = 0; q < (RJ + 1) / 2; ++q) p[e][q] = 0u;
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t af[4] = {x0[s], x1[s], x0[4 + s], x1[4 + s]};
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          const uint32_t bf[2] = {pair_halves(p[2 * s][j / 2], p[2 * s + 1][j / 2], j % 2),
                                  pair_halves(p[8 + 2 * s][j / 2], p[9 + 2 * s][j / 2], j % 2)};
          mma_16816(acc[j], af, bf);
        }
      }
    }
  }
  // D: rows g, g + 8, columns 2 t, 2 t + 1 of tile j
#pragma unroll
  for (int j = 0; j < RJ; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int col = 2 * t + (q & 1);
      red[warp][g + 8 * (q >> 1)][BY_ROWS ? 8 * j + col : RJ * col + j] = acc[j][q];
    }
  __syncthreads();
  const float f = scale ? ld_f32(scale + adapter) : 1.f;
  if (KS == 1) {
    for (int e = threadIdx.x; e < kTileRows * R; e += kThreads) {
      const int m = ld_int(rows + e / R);
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += red[w][e / R][e % R];
      if (m >= 0) out[(size_t)m * R + e % R] = f * s;
    }
    return;
  }
  // every CTA of the cluster has started (arrived above): remote stores are safe
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  for (int e = threadIdx.x; e < kTileRows * R; e += kThreads) {
    const int row = e / R, j = e % R;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += red[w][row][j];
    const int owner = ((row + 1) * KS - 1) / kTileRows;   // the rank with owner 16 / KS <= row
    *cluster.map_shared_rank(&recv[ks][row - owner * kTileRows / KS][j], owner) = s;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int rbeg = ks * kTileRows / KS, rend = (ks + 1) * kTileRows / KS;
  for (int e = threadIdx.x; e < (rend - rbeg) * R; e += kThreads) {
    const int m = ld_int(rows + rbeg + e / R);
    float s = 0.f;
    for (int q = 0; q < KS; ++q) s += recv[q][e / R][e % R];
    if (m >= 0) out[(size_t)m * R + e % R] = f * s;
  }
}

// ---------------------------------------------------------------- up
// out[m][c] = fp16(res[m][c] + f sum_j q[m][j] P(c, j)): P(c, j) = proj[c][j] when
// BY_ROWS (B [N, r]), proj[j][c] else (A [r, K]).  Tokens without an adapter get
// their residual, or zeros.
//
// A warp has one tile's 16 tokens and blocks of 64 columns.  Column 8 n + i of a
// block is column n of tensor-core tile i, so that a lane's results are 16
// consecutive columns of its two rows: it reads the residual and writes the output,
// and by columns also the matrix, in 16-byte vectors, and nothing goes through
// shared memory.
template <bool BY_ROWS, int RJ>
__global__ void __launch_bounds__(kThreads)
q4gsw_adapters_up_kernel(const float* inter, const __half* proj,
                         const float* scale, const int32_t* plan, const __half* res, __half* out, int M,
                         int L, int C, int tile_warps, int blocks_per_warp) {
  constexpr int R = 8 * RJ;
  constexpr int KT = (RJ + 1) / 2;    // tensor-core steps of 16 ranks
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
  const int ma = ld_int(P.rows + (size_t)slot * kTileRows + g), mb = ld_int(P.rows + (size_t)slot * kTileRows + g + 8);
  const float f = adapter >= 0 && scale ? ld_f32(scale + adapter) : 1.f;
  // The intermediate's fragments: rank 2 RJ t + e of a lane, e = 4 s .. 4 s + 3 in
  // step s (indices 2 t, 2 t + 1, 2 t + 8, 2 t + 9); two fp16 parts, hi and lo, of
  // the row over 2^k, k the exponent of its largest value.
  uint32_t hi[KT][4], lo[KT][4];
  float back[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int m = h ? mb : ma;
    float v[4 * KT];
#pragma unroll
    for (int e = 0; e < 4 * KT; ++e) v[e] = 0.f;
    if (m >= 0 && adapter >= 0) {
      const float2* src = reinterpret_cast<const float2*>(inter + (size_t)m * R + 2 * RJ * t);
#pragma unroll
      for (int e = 0; e < RJ; ++e) {
        const uint2 w = ld_v2(src + e);
        v[2 * e] = __uint_as_float(w.x);
        v[2 * e + 1] = __uint_as_float(w.y);
      }
    }
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
  const __half* mat = proj + (size_t)(adapter < 0 ? 0 : adapter) * R * C;
  for (int b = first; b < last; ++b) {
    const int base = 64 * b;
    float acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][q] = 0.f;
    if (adapter >= 0) {
      const bool in = base + 8 * g < C;     // C % 8 == 0
      if constexpr (BY_ROWS) {
        uint32_t w[8][RJ];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (in) {
            load_bytes<4 * RJ>(w[i], mat + (size_t)(base + 8 * g + i) * R + 2 * RJ * t);
          } else {
#pragma unroll
            for (int e = 0; e < RJ; ++e) w[i][e] = 0u;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int s = 0; s < KT; ++s) {
            const uint32_t bf[2] = {w[i][2 * s], 2 * s + 1 < RJ ? w[i][2 * s + 1 < RJ ? 2 * s + 1 : 0] : 0u};
            mma_16816(acc[i], lo[s], bf);
            mma_16816(acc[i], hi[s], bf);
          }
      } else {
#pragma unroll
        for (int s = 0; s < KT; ++s) {
          uint4 w[4];     // ranks 4 s .. 4 s + 3 of the lane, 8 columns each
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = in && 4 * s + e < 2 * RJ ? ld_v4(mat + (size_t)(2 * RJ * t + 4 * s + e) * C + base + 8 * g)
                                            : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&w[0]);
          const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&w[1]);
          const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&w[2]);
          const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&w[3]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t bf[2] = {pair_halves(w0[i / 2], w1[i / 2], i % 2), pair_halves(w2[i / 2], w3[i / 2], i % 2)};
            mma_16816(acc[i], lo[s], bf);
            mma_16816(acc[i], hi[s], bf);
          }
        }
      }
    }
    // columns base + 16 t + i (acc[i][0], row g; [2], row g + 8) and + 8 + i ([1], [3])
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = h ? mb : ma;
      if (m < 0) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = base + 16 * t + 8 * e;
        if (c >= C) continue;
        const size_t at = (size_t)m * C + c;
        uint4 r = make_uint4(0u, 0u, 0u, 0u);
        if (res) r = *reinterpret_cast<const uint4*>(res + at);
        const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 rf = __half22float2(u32_as_h2(rw[i]));
          o[i] = adapter < 0 ? rw[i]
                             : h2_as_u32(__floats2half2_rn(fmaf(back[h], acc[2 * i][2 * h + e], rf.x),
                                                           fmaf(back[h], acc[2 * i + 1][2 * h + e], rf.y)));
        }
        *reinterpret_cast<uint4*>(out + at) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
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
  static constexpr int CW = MT <= 2 ? 64 : 32;     // columns of a block: at most 64 sums a lane
  static constexpr int V = CW / 8;                 // columns of a lane
};

template <bool BY_ROWS, int RJ>
__global__ void __launch_bounds__(kThreads)
q4gsw_adapters_grad_kernel(const __half* act, const float* q,
                           const float* scale, const int32_t* plan, float* out, int M, int L,
                           int C, int accumulate) {
  using T = GradTile<RJ>;
  constexpr int R = 8 * RJ, MT = T::MT, CW = T::CW, V = T::V;
  __shared__ float red[kWarps / 2][MT * V * 4][32];
  griddep_launch_dependents();
  griddep_wait();
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int adapter = blockIdx.y;
  const int base = CW * blockIdx.x;
  const int begin = ld_int(P.first + adapter), end = ld_int(P.first + adapter + 1);
  float acc[MT][V][4];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[a][i][k] = 0.f;
  const int col = base + V * g;
  const bool in = col < C;        // C % 8 == 0, V is 4 or 8
  for (int p0 = begin + 8 * warp; p0 < end; p0 += 8 * kWarps) {
    uint32_t hi[MT][4], lo[MT][4];
    uint32_t x[2][V / 2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = p0 + t + 4 * h;
      const int m = p < end ? ld_int(P.order + p) : -1;
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = 16 * a + g + 8 * k;
          const float w = m >= 0 && j < R ? ld_f32(q + (size_t)m * R + j) : 0.f;
          hi[a][2 * h + k] = to_tf32(w);
          lo[a][2 * h + k] = to_tf32(w - __uint_as_float(hi[a][2 * h + k]));
        }
      if (m >= 0 && in) {
        load_bytes<2 * V>(x[h], act + (size_t)m * C + col);
      } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) x[h][i] = 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 f0 = __half22float2(u32_as_h2(x[0][i / 2])), f1 = __half22float2(u32_as_h2(x[1][i / 2]));
      const uint32_t b0 = __float_as_uint(i % 2 ? f0.y : f0.x), b1 = __float_as_uint(i % 2 ? f1.y : f1.x);
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        mma_1688_tf32(acc[a][i], lo[a], b0, b1);
        mma_1688_tf32(acc[a][i], hi[a], b0, b1);
      }
    }
  }
  // the warps' sums, halves at a time
#pragma unroll
  for (int n = kWarps / 2; n >= 1; n /= 2) {
    if (warp >= n && warp < 2 * n) {
#pragma unroll
      for (int e = 0; e < MT * V * 4; ++e) red[warp - n][e][lane] = acc[e / (V * 4)][e / 4 % V][e % 4];
    }
    __syncthreads();
    if (warp < n) {
#pragma unroll
      for (int e = 0; e < MT * V * 4; ++e) acc[e / (V * 4)][e / 4 % V][e % 4] += red[warp][e][lane];
    }
    __syncthreads();
  }
  if (warp) return;
  if (accumulate && begin == end) return;
  const float f = scale ? ld_f32(scale + adapter) : 1.f;
  float* dst = out + (size_t)adapter * R * C;
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = 16 * a + g + 8 * (k >> 1), c = base + V * (2 * t + (k & 1)) + i;
        if (j >= R || c >= C) continue;
        float* at = BY_ROWS ? dst + (size_t)c * R + j : dst + (size_t)j * C + c;
        *at = accumulate ? fmaf(f, acc[a][i][k], *at) : f * acc[a][i][k];
      }
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

cudaError_t launch_adapters_down(const AdaptersRef& ad, const uint16_t* act, bool by_rows, const uint16_t* proj,
                                 const float* scale, int M, int C, float* out, cudaStream_t stream) {
  // contraction splits: about two CTAs per SM, a chunk of 64 columns per warp, clusters of at most 8
  const int slots = ma::plan_slots(M, ad.L);
  const int chunks = (C + 63) / 64;
  int KS = (2 * sm_count(current_device()) + slots - 1) / slots;
  KS = KS > 8 ? 8 : KS;
  while (KS > 1 && chunks / KS < ma::kWarps) --KS;
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
  const __half* a = reinterpret_cast<const __half*>(act);
  const __half* p = reinterpret_cast<const __half*>(proj);
#define Q4_DOWN(RJ_)                                                                                              \
  return by_rows ? cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_down_kernel<true, RJ_>, a, p, scale, ad.plan, out, M, \
                                      ad.L, C)                                                                    \
                 : cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_down_kernel<false, RJ_>, a, p, scale, ad.plan, out, M, \
                                      ad.L, C)
  Q4_RANKS(ad.r / 8, Q4_DOWN)
#undef Q4_DOWN
}

cudaError_t launch_adapters_up(const AdaptersRef& ad, const float* inter, bool by_rows, const uint16_t* proj,
                               const float* scale, int M, int C, const uint16_t* res, uint16_t* out,
                               cudaStream_t stream) {
  const int slots = ma::plan_slots(M, ad.L);
  int tile_warps = 1;
  while (tile_warps < ma::kWarps && tile_warps < slots) tile_warps *= 2;
  const int col_warps = ma::kWarps / tile_warps;
  const int blocks = (C + 63) / 64, groups = (slots + tile_warps - 1) / tile_warps;
  const int per = 1;
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

cudaError_t launch_adapters_grad(const AdaptersRef& ad, const uint16_t* act, const float* q, bool by_rows,
                                 const float* scale, int M, int C, bool accumulate, float* out, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(ma::kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  serialize(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const __half* a = reinterpret_cast<const __half*>(act);
#define Q4_GRAD(RJ_)                                                                                              \
  cfg.gridDim = dim3((C + ma::GradTile<RJ_>::CW - 1) / ma::GradTile<RJ_>::CW, ad.L, 1);                           \
  return by_rows ? cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_grad_kernel<true, RJ_>, a, q, scale, ad.plan, out, M, \
                                      ad.L, C, (int)accumulate)                                                   \
                 : cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_grad_kernel<false, RJ_>, a, q, scale, ad.plan, out, M, \
                                      ad.L, C, (int)accumulate)
  Q4_RANKS(ad.r / 8, Q4_GRAD)
#undef Q4_GRAD
}

}  // namespace q4gsw
