// q4gsw_adapters.cu - the low-rank half of a projection with an adapter for
// every token, and the gradients of the adapters (sm_100a).
//
// Over the tiles of a plan (16 tokens of one adapter each):
//   down   u = x A^T (forward), v = s d_y B (backward): the intermediate, fp32 [M][r]
//   up     the low-rank term s u B^T (or v A) with the residual, fp16 [M][C], left in
//          the output's place: the base product then adds itself as to any residual
//   low    both in one launch, for few tiles
//   grad   d_A = v^T x, d_B = s d_y^T u over the tokens of each adapter, fp32
// so that the base product runs on its own routes unchanged, at any number of tokens
// and with either kind of scales.  The first kernel lets the next start only behind its
// own wait; the product, launched behind them, then knows its activations to be
// complete, reads them at once and waits for the low-rank term in its epilogue alone: one
// token of 8192 x 2048 takes 7.3 us (10.4 with two kernels in a row in front of it and a
// product that waits for them).
//
// The intermediate stays in fp32: rounded to fp16 it would put 2^-11 of error into
// fp32 gradients, and small gradients would fall below fp16's range.  It goes to the
// tensor cores as two fp16 parts over a power of two near the largest value of the
// token's row (`up`) or of the rank's chunk of tokens (`grad`): 2^-23 of that is lost.
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

// 16 bytes to shared memory, zeros where !in (nothing is read then).
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t shared_address(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// Four 8 x 8 matrices of fp16: lanes 8 i .. 8 i + 7 give the rows of matrix i.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

// halves i of two registers: (lo.half[i], hi.half[i])
__device__ __forceinline__ uint32_t pair_halves(uint32_t lo, uint32_t hi, int i) {
  return prmt(lo, hi, i ? 0x7632u : 0x5410u);
}

// The exponent k of a float's pattern (2^k <= |v| < 2^(k + 1)), held where 2^k and 2^-k
// are both normal numbers.
__device__ __forceinline__ int exponent_of(uint32_t bits) {
  const int k = (int)(bits >> 23 & 255u) - 127;
  return max(-126, min(k, 126));
}

constexpr unsigned int kPlanErrorBit = 0x100u;      // as an index out of range

// Whether the plan is one of M tokens over L adapters; the first kernel of a call
// records that it is not.  Looked at before anything else of the plan is read: the
// parts of a plan lie where M and L say, and a plan of fewer tokens ends before them.
__device__ __forceinline__ bool plan_fits(const PlanView& P, int M, int L, unsigned int* error = nullptr) {
  const uint4 h = ld_v4(P.head);
  const bool fits = (int)h.y == M && (int)h.z == L && (int)h.w == kPlanMark;
  if (!fits && error && threadIdx.x == 0) atomicOr(error, kPlanErrorBit);
  return fits;
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
// Their sums are added to acc in fp32 registers (the tensor cores truncate theirs).
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
    float sum[RJ][4];
#pragma unroll
    for (int j = 0; j < RJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[j][e] = 0.f;
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
          mma_16816(sum[j], af, bf);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] += sum[j][e];
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
// is given) of the tile's adapter, for many tiles (few: q4gsw_adapters_low_kernel).
//
// A CTA has a pair of tiles of one adapter, four warps to a tile.  Stages of 128 columns
// of the tiles' tokens and of the adapter's matrix go through a ring in shared memory
// (cp.async), from which the warps take their fragments by ldmatrix: the matrix is read
// once a CTA.  The warps of a tile and the KS CTAs of the cluster (grid = (pairs, KS))
// split the contraction; sums go to fp32 registers every few stages (the tensor cores
// truncate theirs), and the warps' and the CTAs' are added in a fixed order.
//
// 4096 tokens of 4096 with 16 adapters of rank 64: 21 us (the bytes alone 6.4); 1021 of
// 14336 with four: 17.5.  Bound by the latency of a stage's steps at 16 warps an SM
// (issue slots 40 % busy, tensor pipe 17 %, DRAM 15 %).  Four tiles to a CTA read the
// matrix half as often and leave too few CTAs (40 us where two took 29), a deeper ring
// gains nothing; fp32 sums at every stage cost 2 us.
constexpr int kDownTiles = 2;
template <bool BY_ROWS, int RJ>
struct DownRing {
  static constexpr int R = 8 * RJ, WT = kDownTiles, WK = kWarps / WT;
  static constexpr int COLS = 128;                                   // columns of a stage
  static constexpr int FLUSH = 4;                                    // stages whose sums stay in the tensor cores
  static constexpr int STAGES = 3;
  // rows of 16-byte chunks, an odd number of them: ldmatrix meets no bank twice
  static constexpr int X_PITCH = 2 * COLS + 16;
  static constexpr int P_ROWS = BY_ROWS ? R : COLS;
  static constexpr int P_CHUNKS = BY_ROWS ? COLS / 8 : RJ;           // of a row
  static constexpr int P_PITCH = BY_ROWS ? X_PITCH : 16 * (RJ | 1);
  static constexpr int X_BYTES = WT * kTileRows * X_PITCH, P_BYTES = P_ROWS * P_PITCH;
  static constexpr int STAGE = X_BYTES + P_BYTES;
  static constexpr int RED = kWarps * kTileRows * R * 4;             // reuses the ring
  static constexpr int RECV = WT * kTileRows * R * 4;
  static constexpr int RING = STAGES * STAGE > RED ? STAGES * STAGE : RED;
  static constexpr int BYTES = RING + RECV;
};

template <bool BY_ROWS, int RJ>
__global__ void __launch_bounds__(kThreads, 2)
q4gsw_adapters_down_kernel(const __half* act, const __half* proj, const float* scale, const int32_t* plan, float* out,
                           int M, int L, int C, unsigned int* error) {
  using D = DownRing<BY_ROWS, RJ>;
  constexpr int R = D::R, WT = D::WT, WK = D::WK;
  extern __shared__ __align__(16) unsigned char down_smem[];
  __shared__ int s_row[WT * kTileRows];
  auto red = reinterpret_cast<float (*)[kTileRows][R]>(down_smem);             // [kWarps]
  auto recv = reinterpret_cast<float (*)[kTileRows][R]>(down_smem + D::RING);   // [WT], [sender][owned row] of each
  const uint32_t ring = shared_address(down_smem);
  griddep_wait();
  griddep_launch_dependents();     // behind the wait: what ran before has been written when the next kernel starts
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  const int KS = gridDim.y, ks = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  if (!plan_fits(P, M, L, error)) return;                   // the whole cluster
  const int slot0 = ld_int(P.pair + blockIdx.x);
  if (slot0 < 0) return;                                    // the whole cluster
  const bool more = slot0 + 1 < plan_slots(M, L);           // (loads that do not wait for one another)
  const int adapter = ld_int(P.tile + slot0), behind = more ? ld_int(P.tile + slot0 + 1) : kNoTile;
  int my_row = -1;
  if (threadIdx.x < (more ? WT : 1) * kTileRows) my_row = ld_int(P.rows + (size_t)slot0 * kTileRows + threadIdx.x);
  if (threadIdx.x < WT * kTileRows) s_row[threadIdx.x] = behind == adapter || threadIdx.x < kTileRows ? my_row : -1;
  __syncthreads();
  if (adapter < 0) {
    for (int e = threadIdx.x + ks * kThreads; e < WT * kTileRows * R; e += KS * kThreads)
      if (s_row[e / R] >= 0) out[(size_t)s_row[e / R] * R + e % R] = 0.f;
    return;
  }
  if (KS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int stages = (C + D::COLS - 1) / D::COLS;
  const int it_begin = (int)((long long)ks * stages / KS), it_end = (int)((long long)(ks + 1) * stages / KS);
  const int my_tile = warp / WK, my_part = warp % WK;
  float total[RJ][4];
#pragma unroll
  for (int j = 0; j < RJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) total[j][e] = 0.f;
  // what this thread copies of a stage: 16 bytes of a row of each tile, and of the matrix rows
  // 16 apart (by rows) or pieces kThreads apart of the stage's contiguous columns
  const int q16 = threadIdx.x % 16, row16 = threadIdx.x / 16;
  const __half* x_from[WT];
#pragma unroll
  for (int i = 0; i < WT; ++i) {
    const int m = s_row[16 * i + row16];
    x_from[i] = m >= 0 ? act + (size_t)m * C + 8 * q16 : nullptr;
  }
  const __half* mat = proj + (size_t)adapter * R * C;
  const __half* p_from = BY_ROWS ? mat + (size_t)row16 * C + 8 * q16 : mat + 8 * threadIdx.x;
  auto issue = [&](int it, uint32_t st) {
    if (it < it_end) {
      const int c0 = it * D::COLS;
      const bool in = c0 + 8 * q16 < C;                       // C % 8 == 0: a chunk is wholly in or out
#pragma unroll
      for (int i = 0; i < WT; ++i) {
        const bool live = in && x_from[i];
        copy_16(st + (16 * i + row16) * D::X_PITCH + 16 * q16, live ? x_from[i] + c0 : act, live);
      }
      const uint32_t sp = st + D::X_BYTES;
      if constexpr (BY_ROWS) {
        const __half* from = in ? p_from + c0 : proj;
        const size_t step = in ? (size_t)16 * C : 0;
#pragma unroll
        for (int i = 0; i < (R + 15) / 16; ++i)
          if (R % 16 == 0 || row16 + 16 * i < R)
            copy_16(sp + (row16 + 16 * i) * D::P_PITCH + 16 * q16, from + i * step, in);
      } else {
        const __half* from = p_from + (size_t)c0 * R;
#pragma unroll
        for (int i = 0; i < (D::P_ROWS * RJ + kThreads - 1) / kThreads; ++i) {
          const int e = threadIdx.x + i * kThreads;
          if (D::P_ROWS * RJ % kThreads && e >= D::P_ROWS * RJ) break;
          const bool live = c0 + e / RJ < C;
          copy_16(sp + e / RJ * D::P_PITCH + 16 * (e % RJ), live ? from + 8 * i * kThreads : proj, live);
        }
      }
    }
    cp_async_commit();
  };
  uint32_t used = ring, filled = ring;      // the stages' places, in turn
  auto next = [&](uint32_t st) { return st + D::STAGE == ring + D::STAGES * D::STAGE ? ring : st + D::STAGE; };
  for (int i = 0; i < D::STAGES - 1; ++i, filled = next(filled)) issue(it_begin + i, filled);
  float acc[RJ][4];
#pragma unroll
  for (int j = 0; j < RJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  for (int it = it_begin; it < it_end; ++it, used = next(used), filled = next(filled)) {
    cp_async_wait<D::STAGES - 2>();
    __syncthreads();                     // the stage has landed, and the one refilled below has been used by all
    issue(it + D::STAGES - 1, filled);
    const uint32_t st = used;
    // rows 0-7, 8-15 at columns 0-7, then both at columns 8-15 of a step of 16
    const uint32_t xa = st + (my_tile * kTileRows + lane % 16) * D::X_PITCH + 16 * (lane / 16);
    const uint32_t pa = st + D::X_BYTES;
#pragma unroll
    for (int k = 0; k < D::COLS / 16 / WK; ++k) {
      const int step = my_part * (D::COLS / 16 / WK) + k;
      uint32_t af[4];
      ldmatrix4(af, xa + 32 * step);
#pragma unroll
      for (int j = 0; j < RJ; j += 2) {
        // ranks 8 j .. 8 j + 15 (the second eight repeat the first where RJ is odd)
        uint32_t bf[4];
        const int jr = j + 1 < RJ ? lane / 16 : 0;
        if constexpr (BY_ROWS)
          ldmatrix4(bf, pa + (8 * (j + jr) + lane % 8) * D::P_PITCH + 32 * step + 16 * (lane / 8 % 2));
        else
          ldmatrix4_trans(bf, pa + (16 * step + lane % 16) * D::P_PITCH + 16 * (j + jr));
        const uint32_t b0[2] = {bf[0], bf[1]}, b1[2] = {bf[2], bf[3]};
        mma_16816(acc[j], af, b0);
        if (j + 1 < RJ) mma_16816(acc[j + 1 < RJ ? j + 1 : j], af, b1);
      }
    }
    if ((it - it_begin) % D::FLUSH == D::FLUSH - 1 || it == it_end - 1) {
#pragma unroll
      for (int j = 0; j < RJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          total[j][e] += acc[j][e];
          acc[j][e] = 0.f;
        }
    }
  }
  cp_async_wait<0>();
  __syncthreads();                       // the ring is free
  down_park<true, RJ>(total, red[warp], g, t);
  __syncthreads();
  // the sums of row `row` of tile `w0` over its warps
  auto own = [&](int w0, int row, int j) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) s += red[w0 * WK + w][row][j];
    return s;
  };
  const int owned = kTileRows / KS;      // rows of each tile that this CTA writes (KS is a power of two)
  if (KS > 1) {
    // every CTA of the cluster has started (arrived above): remote stores are safe
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    for (int e = threadIdx.x; e < WT * kTileRows * R; e += kThreads) {
      const int w = e / (kTileRows * R), row = e / R % kTileRows, j = e % R;
      *cluster.map_shared_rank(&recv[w][ks * owned + row % owned][j], row / owned) = own(w, row, j);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  for (int e = threadIdx.x; e < WT * owned * R; e += kThreads) {
    const int w = e / (owned * R), row = e / R % owned, j = e % R;
    const int m = s_row[w * kTileRows + ks * owned + row];
    if (m < 0) continue;
    float v = 0.f;
    if (KS > 1) {
      for (int q = 0; q < KS; ++q) v += recv[w][q * owned + row][j];
    } else {
      v = own(w, row, j);
    }
    out[(size_t)m * R + j] = scale ? ld_f32(scale + adapter) * v : v;
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
// side, and nothing goes through shared memory (few tiles: up_block).

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
      const int k = exponent_of(__float_as_uint(top));     // an infinite or NaN value stays what it is
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

// The same for many tiles.  A CTA has two pairs of tiles, a tile to a warp, and a run of
// column blocks, whose part of the matrices of the one or two adapters goes through a
// ring in shared memory: it is read once for 64 (or 32) tokens, and its fragments come by
// ldmatrix (in their natural order).  Sums are turned in shared memory, so that rows are
// read (the residual) and written in whole lines: as fp16 where there is no residual, else
// in fp32, to which it is added before the one rounding.
//
// 4096 x 14336, rank 64, no residual: 49.5 us (60 with every turn in fp32 and a third
// stage, which left three CTAs an SM; the writes alone 18).  The two parts keep the tensor
// pipe half busy; the rest is latency that 16 warps an SM do not cover.
constexpr int kUpWarps = 4, kUpThreads = 32 * kUpWarps;
template <bool BY_ROWS, int RJ>
struct UpRing {
  static constexpr int R = 8 * RJ, KT = (RJ + 1) / 2;
  static constexpr int STAGES = 2;
  static constexpr int ROWS = BY_ROWS ? 64 : 16 * KT;                // rows of a block (ranks padded to 16)
  static constexpr int CHUNKS = BY_ROWS ? 2 * KT : 8;                // 16-byte chunks of a row
  static constexpr int PITCH = 16 * (CHUNKS + 1);                    // an odd number of them
  static constexpr int REGION = ROWS * PITCH, STAGE = 2 * REGION;
  static constexpr int T_PITCH = 72;                                 // of a warp's 16 x 64 sums, floats
  static constexpr int BYTES = STAGES * STAGE + kUpWarps * kTileRows * T_PITCH * 2;    // without a residual: as fp16
  static constexpr int BYTES_RES = STAGES * STAGE + kUpWarps * kTileRows * T_PITCH * 4;
};

template <bool BY_ROWS, int RJ>
__global__ void __launch_bounds__(kUpThreads, 4)
q4gsw_adapters_up_kernel(const float* inter, const __half* proj, const float* scale, const int32_t* plan,
                         const __half* res, __half* out, int M, int L, int C, int blocks_per_cta) {
  using U = UpRing<BY_ROWS, RJ>;
  constexpr int R = U::R, KT = U::KT;
  extern __shared__ __align__(16) unsigned char up_smem[];
  griddep_launch_dependents();
  griddep_wait();
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // the two pairs' first tiles, their adapters, and this warp's tile
  if (!plan_fits(P, M, L)) return;
  const int pairs = plan_pairs(M, L);
  const int s0 = ld_int(P.pair + 2 * blockIdx.x), s1 = 2 * (int)blockIdx.x + 1 < pairs ? ld_int(P.pair + 2 * blockIdx.x + 1) : -1;
  if (s0 < 0) return;                              // pairs in use come first
  const int a0 = ld_int(P.tile + s0), a1 = s1 >= 0 ? ld_int(P.tile + s1) : kNoTile;
  const int base_slot = warp < 2 ? s0 : s1, theirs = warp < 2 ? a0 : a1;
  const bool there = base_slot >= 0 && base_slot + (warp & 1) < plan_slots(M, L);
  const int slot = there ? base_slot + (warp & 1) : s0;      // (loads that do not wait for one another)
  const int its = ld_int(P.tile + slot);
  const int32_t* rows = P.rows + (size_t)slot * kTileRows;
  int m[2] = {ld_int(rows + g), ld_int(rows + g + 8)};
  // rows 4 k + lane / 8 of the tile, columns 8 (lane % 8) .. of a block: what the lane writes
  int to[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) to[k] = ld_int(rows + 4 * k + lane / 8);
  const int mine = there && its == theirs ? its : kNoTile;
  if (mine == kNoTile) m[0] = m[1] = to[0] = to[1] = to[2] = to[3] = -1;
  const int first = blockIdx.y * blocks_per_cta, last = min(first + blocks_per_cta, (C + 63) / 64);
  const uint32_t ring = shared_address(up_smem);
  const bool other = a1 >= 0 && a1 != a0;  // a second matrix, in the second region
  const uint32_t region = mine == a1 && other ? (uint32_t)U::REGION : 0u;
  auto issue = [&](int b) {
    if (b < last) {
      const uint32_t st = ring + (uint32_t)((b - first) % U::STAGES) * U::STAGE;
      for (int e = threadIdx.x; e < U::ROWS * U::CHUNKS; e += kUpThreads) {
        const int row = e / U::CHUNKS, k = e % U::CHUNKS;
        // by rows: column 64 b + row, ranks 8 k ..; else rank row, columns 64 b + 8 k ..
        const bool in = BY_ROWS ? 64 * b + row < C && k < RJ : row < R && 64 * b + 8 * k < C;
        const size_t from = BY_ROWS ? (size_t)(64 * b + row) * R + 8 * k : (size_t)row * C + 64 * b + 8 * k;
        const uint32_t to_smem = st + row * U::PITCH + 16 * k;
        copy_16(to_smem, proj + (in ? (size_t)a0 * R * C + from : 0), in);
        if (other) copy_16(to_smem + U::REGION, proj + (in ? (size_t)a1 * R * C + from : 0), in);
      }
    }
    cp_async_commit();
  };
  if (a0 >= 0)
    for (int i = 0; i < U::STAGES - 1; ++i) issue(first + i);
  UpTile<RJ> q;
  // ranks 16 s + 2 t, + 1, + 8, + 9 of the lane in step s
  q.fill(mine >= 0 && scale ? ld_f32(scale + mine) : 1.f, [&](int h, int e, float& v0, float& v1) {
    if (m[h] < 0 || mine < 0) return;
    const uint2 w = ld_v2(inter + (size_t)m[h] * R + 16 * (e / 4) + 4 * (e % 4) + 2 * t);
    v0 = __uint_as_float(w.x);
    v1 = __uint_as_float(w.y);
  });
  float* turn = reinterpret_cast<float*>(up_smem + U::STAGES * U::STAGE) + warp * kTileRows * U::T_PITCH;
  __half* turn_half = reinterpret_cast<__half*>(up_smem + U::STAGES * U::STAGE) + warp * kTileRows * U::T_PITCH;
  auto write = [&](int b, bool sums) {
    const int c = 64 * b + 8 * (lane % 8);
    if (c >= C) return;                    // C % 8 == 0
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (to[k] < 0) continue;
      const size_t at = (size_t)to[k] * C + c;
      uint4 r = make_uint4(0u, 0u, 0u, 0u);
      if (res) r = *reinterpret_cast<const uint4*>(res + at);
      if (sums) {
        // (the upper four of eight lanes read their halves in the other order: no bank twice)
        const float* v = turn + (4 * k + lane / 8) * U::T_PITCH + 8 * (lane % 8);
        const bool up = lane & 4;
        const float4 p = *reinterpret_cast<const float4*>(v + (up ? 4 : 0)),
                     q2 = *reinterpret_cast<const float4*>(v + (up ? 0 : 4));
        const float4 v0 = up ? q2 : p, v1 = up ? p : q2;
        const float2 r0 = __half22float2(u32_as_h2(r.x)), r1 = __half22float2(u32_as_h2(r.y)),
                     r2 = __half22float2(u32_as_h2(r.z)), r3 = __half22float2(u32_as_h2(r.w));
        r = make_uint4(h2_as_u32(__floats2half2_rn(v0.x + r0.x, v0.y + r0.y)),
                       h2_as_u32(__floats2half2_rn(v0.z + r1.x, v0.w + r1.y)),
                       h2_as_u32(__floats2half2_rn(v1.x + r2.x, v1.y + r2.y)),
                       h2_as_u32(__floats2half2_rn(v1.z + r3.x, v1.w + r3.y)));
      }
      *reinterpret_cast<uint4*>(out + at) = r;
    }
  };
  if (mine == kNoAdapter)                  // the residual, or zeros
    for (int b = first; b < last; ++b) write(b, false);
  if (a0 < 0) return;                      // (sorted: the second pair has no adapter, either)
  for (int b = first; b < last; ++b) {
    cp_async_wait<U::STAGES - 2>();
    __syncthreads();                     // the block has landed, and the one refilled below has been used by all
    issue(b + U::STAGES - 1);
    if (mine < 0) continue;
    const uint32_t st = ring + (uint32_t)((b - first) % U::STAGES) * U::STAGE + region;
    float acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
    for (int s = 0; s < KT; ++s) {
      uint32_t bf[4][4];                 // columns 16 i .. + 7 (indices 0-7, 8-15), then + 8 .. + 15
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BY_ROWS)
          ldmatrix4(bf[i], st + (16 * i + 8 * (lane / 16) + lane % 8) * U::PITCH + 32 * s + 16 * (lane / 8 % 2));
        else
          ldmatrix4_trans(bf[i], st + (16 * s + lane % 16) * U::PITCH + 32 * i + 16 * (lane / 16));
      }
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t f[2] = {bf[i / 2][2 * (i % 2)], bf[i / 2][2 * (i % 2) + 1]};
          mma_16816(acc[i], part ? q.hi[s] : q.lo[s], f);
        }
    }
    __syncwarp();                        // the lanes have read the block before
    if (!res) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<uint32_t*>(turn_half + (g + 8 * h) * U::T_PITCH + 8 * i + 2 * t) =
              h2_as_u32(__floats2half2_rn(q.back[h] * acc[i][2 * h], q.back[h] * acc[i][2 * h + 1]));
      __syncwarp();
      const int c = 64 * b + 8 * (lane % 8);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (to[k] >= 0 && c < C)
          *reinterpret_cast<uint4*>(out + (size_t)to[k] * C + c) =
              *reinterpret_cast<const uint4*>(turn_half + (4 * k + lane / 8) * U::T_PITCH + 8 * (lane % 8));
      continue;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(turn + (g + 8 * h) * U::T_PITCH + 8 * i + 2 * t) =
            make_float2(q.back[h] * acc[i][2 * h], q.back[h] * acc[i][2 * h + 1]);
    __syncwarp();
    write(b, true);
  }
  cp_async_wait<0>();                      // no thread leaves with copies in flight
}

// ---------------------------------------------------------------- down and up in one
// For few tiles: a cluster of KS CTAs has one tile.  Its CTAs split the contraction of
// `down`, each gets the sums of all of them (every CTA writes its own to every other's
// shared memory, added in rank order), and they split the columns of `up`.  One launch
// and one exchange in place of two launches and a trip through memory; `inter` is
// written for the backward pass.  FWD: x, A, B; else d_y, B, A.
//
// 512 tokens of 8 adapters, rank 16, 2048 <-> 8192: 8.7 us, of which the launch, the plan
// and the exchange are five; bound by latency (a chain of loads, the exchange, loads).
// W warps: eight, or four beside the product of up to 16 tokens (launch_adapters_low).
template <bool FWD, int RJ, int U, int W>
__global__ void __launch_bounds__(32 * W, W == 4 && RJ <= 2 ? (U == 1 ? 6 : 4) : U == 1 && RJ <= 2 ? 3 : 1)
q4gsw_adapters_low_kernel(const __half* act, const __half* mat_down, const __half* mat_up, const float* scale,
                          const int32_t* plan, float* inter, const __half* res, __half* out, int M, int L, int C_down,
                          int C_up, unsigned int* error) {
  constexpr int R = 8 * RJ;
  extern __shared__ __align__(16) float low_smem[];
  auto red = reinterpret_cast<float (*)[kTileRows][R]>(low_smem);                       // [W]
  auto recv = reinterpret_cast<float (*)[kTileRows][R]>(low_smem + W * kTileRows * R);   // [KS], by sender
  griddep_wait();
  griddep_launch_dependents();     // behind the wait: what ran before has been written when the next kernel starts
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  const int KS = gridDim.y, ks = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  if (!plan_fits(P, M, L, error)) return;
  const int adapter = ld_int(P.tile + blockIdx.x);
  const int32_t* rows = P.rows + (size_t)blockIdx.x * kTileRows;
  const int m[2] = {ld_int(rows + g), ld_int(rows + g + 8)};
  if (adapter == kNoTile) return;
  UpTile<RJ> q;
  const __half* up = mat_up + (size_t)(adapter < 0 ? 0 : adapter) * R * C_up;
  const int blocks = out ? (C_up + 63) / 64 : 0;      // without an output: the intermediate alone
  if (adapter >= 0) {
    if (KS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    // the first block's part of `up`'s matrix on its way to L2 meanwhile
    const int b0 = ks * W + warp;
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
    const int chunks = (C_down + 63) / 64, parts = KS * W, part = ks * W + warp;
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
      for (int e = threadIdx.x; e < kTileRows * R; e += 32 * W) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += red[w][e / R][e % R];
        for (int k = 0; k < KS; ++k) *cluster.map_shared_rank(&recv[ks][e / R][e % R], k) = s;
      }
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    const float f = scale ? ld_f32(scale + adapter) : 1.f;
    for (int e = threadIdx.x; e < kTileRows * R; e += 32 * W) {
      float s = 0.f;
      if (KS > 1) {
        for (int k = 0; k < KS; ++k) s += recv[k][e / R][e % R];
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) s += red[w][e / R][e % R];
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
    for (int e = threadIdx.x; e < kTileRows * R; e += 32 * W) {
      const int to = ld_int(rows + e / R);
      if (to >= 0) inter[(size_t)to * R + e % R] = 0.f;
    }
  }
  for (int b = ks * W + warp; b < blocks; b += KS * W)
    up_block<FWD, RJ>(up, q, adapter >= 0, m, 64 * b, C_up, res, out, g, t);
}

// ---------------------------------------------------------------- grad
// G_a(c, j) = f sum over the tokens m of adapter a of act[m][c] q[m][j], fp32, as
// rows [c][r] (BY_ROWS: d_B [N, r]) or [r][c] (d_A [r, K]).  f the adapter's factor
// (scale given) or 1.
//
// A CTA has W columns of one adapter, its warps CW each and all ranks (half of them from 56 on).  Chunks of 32
// tokens (their columns, and their rows of q) go through a ring in shared memory; each
// rank's q of a chunk is divided by a power of two near its largest value and split
// into two fp16 parts, once for all warps, and the chunk's sums are scaled back when
// they are added to the fp32 registers: 2^-23 of the largest q of the chunk is lost, no
// range, and the tensor cores' own sums are two steps long.  The Z CTAs of a cluster
// take every Z-th chunk, and their sums are added through distributed shared memory in
// rank order.
//
// 1021 tokens of four adapters, 4096 and 14336 columns, rank 64: 24.2 us (the bytes alone
// 8.6); 512 of eight, 8192 and 2048, rank 16: 8.7.  Bound by the steps of a chunk (three
// barriers, the split, then the products: issue slots 44 % busy, tensor pipe 25 %).  With
// all ranks to every warp 26.7; chunks of 64 tokens, CTAs of 512 threads and tf32
// products were slower (47.5 against 43.5, 40 against 29, 43 against 28).
// Up to rank 16 three CTAs an SM: 128 adapters of one token each, 4096 and 4096, 38.6 ->
// 31.4 us; rank 32 in 80 registers gains 7 % there and loses 5 % with six adapters.
constexpr int kChunk = 32;      // tokens

template <int RJ>
struct GradTile {
  static constexpr int R = 8 * RJ, MT = (RJ + 1) / 2;                // tensor-core tiles of 16 ranks
  static constexpr int RW = MT == 4 ? 2 : 1, WT = MT / RW;            // warps beside each other over the ranks, tiles of each
  static constexpr int CW = MT == 3 ? 16 : 32;                       // columns of a warp
  static constexpr int W = kWarps / RW * CW;
  static constexpr int STAGES = 3;
  static constexpr int X_PITCH = 2 * W + 16;                         // an odd number of 16-byte chunks
  static constexpr int X_BYTES = kChunk * X_PITCH, Q_BYTES = kChunk * R * 4;
  static constexpr int STAGE = X_BYTES + Q_BYTES;
  static constexpr int H_PITCH = 2 * 16 * MT + 16;                   // rows of the two parts, ranks padded to 16
  static constexpr int H_BYTES = kChunk * H_PITCH;
  static constexpr int SUMS = (W + 4) * R * 4 > W * (R + 4) * 4 ? (W + 4) * R * 4 : W * (R + 4) * 4;   // reuses the ring
  static constexpr int RING = STAGES * STAGE > SUMS ? STAGES * STAGE : SUMS;
  static constexpr int BYTES = RING + 2 * H_BYTES;
};

// One of the two gradients: the columns' activations and the other factor.
struct GradSide {
  const __half* act;
  const float* q;
  const float* scale;
  float* out;
  int C;
};

template <bool BY_ROWS, int RJ>
__device__ __forceinline__ void grad_block(const GradSide& a, const PlanView& P, int group, int accumulate,
                                           unsigned char* smem, unsigned int* s_top) {
  using T = GradTile<RJ>;
  constexpr int R = T::R, WT = T::WT, CW = T::CW, W = T::W;
  constexpr int PITCH = (BY_ROWS ? R : W) + 4;        // of the sums in shared memory, floats
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) / T::RW;      // of the columns
  const int rank0 = 16 * WT * ((threadIdx.x >> 5) % T::RW);                  // this warp's ranks
  const int g = lane >> 2, t = lane & 3;
  const int adapter = blockIdx.y, Z = gridDim.z, z = blockIdx.z;
  const int base = W * group;
  const int begin = ld_int(P.first + adapter), end = ld_int(P.first + adapter + 1);
  float* dst = a.out + (size_t)adapter * R * a.C;
  if (begin == end) {                                 // no tokens: zeros (the whole cluster leaves here)
    if (accumulate) return;
    for (int e = threadIdx.x + z * kThreads; e < W * R / 4; e += Z * kThreads) {
      const int row = BY_ROWS ? e / (R / 4) : e / (W / 4), x4 = BY_ROWS ? e % (R / 4) : e % (W / 4);
      if ((BY_ROWS ? base + row : base + 4 * x4) < a.C)
        *reinterpret_cast<float4*>(BY_ROWS ? dst + (size_t)(base + row) * R + 4 * x4
                                           : dst + (size_t)row * a.C + base + 4 * x4) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  const uint32_t ring = shared_address(smem), parts = ring + T::RING;
  float* sums = reinterpret_cast<float*>(smem);
  const int chunks = (end - begin + kChunk - 1) / kChunk;
  const int mine = chunks > z ? (chunks - z + Z - 1) / Z : 0;      // chunks z, z + Z, ..
  float total[WT][CW / 8][4];
#pragma unroll
  for (int m = 0; m < WT; ++m)
#pragma unroll
    for (int i = 0; i < CW / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) total[m][i][k] = 0.f;
  // the tokens whose rows this thread copies: rows threadIdx.x / XT + k of the columns,
  // and of q; looked up a chunk ahead of their copies
  constexpr int XC = W / 8, XT = kThreads / XC, XN = kChunk / XT;       // chunks of a row, rows at once, rounds
  constexpr int QC = R / 4, QN = (kChunk * QC + kThreads - 1) / kThreads;
  int xt[XN], qt[QN];
  auto look_up = [&](int u) {
    const int p0 = begin + (z + u * Z) * kChunk;
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int p = p0 + (int)threadIdx.x / XC + i * XT;
      xt[i] = u < mine && p < end ? ld_int(P.order + p) : -1;
    }
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int e = threadIdx.x + i * kThreads, p = p0 + e / QC;
      qt[i] = u < mine && e < kChunk * QC && p < end ? ld_int(P.order + p) : -1;
    }
  };
  auto issue = [&](int u) {
    if (u < mine) {
      const uint32_t st = ring + (uint32_t)(u % T::STAGES) * T::STAGE;
      const int k = threadIdx.x % XC, c = base + 8 * k;
#pragma unroll
      for (int i = 0; i < XN; ++i) {
        const bool in = xt[i] >= 0 && c < a.C;        // C % 8 == 0
        copy_16(st + (threadIdx.x / XC + i * XT) * T::X_PITCH + 16 * k, a.act + (in ? (size_t)xt[i] * a.C + c : 0), in);
      }
#pragma unroll
      for (int i = 0; i < QN; ++i) {
        const int e = threadIdx.x + i * kThreads;
        if (e < kChunk * QC)
          copy_16(st + T::X_BYTES + 16 * e, a.q + (qt[i] >= 0 ? (size_t)qt[i] * R + 4 * (e % QC) : 0), qt[i] >= 0);
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < T::STAGES - 1; ++i) {
    look_up(i);
    issue(i);
  }
  look_up(T::STAGES - 1);
  if (R % 16) {      // ranks past an odd eight stay zero in the parts
    for (int e = threadIdx.x; e < 2 * kChunk * 8; e += kThreads)
      *reinterpret_cast<__half*>(smem + T::RING + (e / 8) * T::H_PITCH + 2 * (R + e % 8)) = __float2half_rn(0.f);
  }
  if (threadIdx.x < R) s_top[threadIdx.x] = 0u;       // of the first chunk
  for (int u = 0; u < mine; ++u) {
    cp_async_wait<T::STAGES - 2>();
    __syncthreads();                     // the chunk has landed; the parts and the stage refilled below have been used
    unsigned int* top = s_top + u % 2 * R;
    if (threadIdx.x < R) s_top[(u + 1) % 2 * R + threadIdx.x] = 0u;
    issue(u + T::STAGES - 1);
    look_up(u + T::STAGES);
    const uint32_t st = ring + (uint32_t)(u % T::STAGES) * T::STAGE;
    const float* q = reinterpret_cast<const float*>(smem + (u % T::STAGES) * T::STAGE + T::X_BYTES);
    // pairs of ranks, RJ / 2 on average to a thread; of one pair where the threads are a
    // multiple of the pairs
    constexpr int PAIRS = kChunk * R / 2, N = (PAIRS + kThreads - 1) / kThreads;
    constexpr bool kOnePair = kThreads % (R / 2) == 0;
    float2 v[N];
    uint32_t most[2] = {0u, 0u};      // (patterns of non-negative floats are ordered as they are; a NaN is above all)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x + i * kThreads;
      if (PAIRS % kThreads && e >= PAIRS) break;
      v[i] = reinterpret_cast<const float2*>(q)[e];
      const uint32_t size[2] = {__float_as_uint(v[i].x) & 0x7fffffffu, __float_as_uint(v[i].y) & 0x7fffffffu};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (kOnePair) most[h] = max(most[h], size[h]);
        else atomicMax(&top[2 * (e % (R / 2)) + h], size[h]);
      }
    }
    if (kOnePair) {
      atomicMax(&top[2 * (threadIdx.x % (R / 2))], most[0]);
      atomicMax(&top[2 * (threadIdx.x % (R / 2)) + 1], most[1]);
    }
    __syncthreads();
    float down[2] = {0.f, 0.f};
    auto look = [&](int e) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        down[h] = __uint_as_float((uint32_t)(127 - exponent_of(top[2 * (e % (R / 2)) + h])) << 23);
    };
    if (kOnePair) look(threadIdx.x);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = threadIdx.x + i * kThreads;
      if (PAIRS % kThreads && e >= PAIRS) break;
      if (!kOnePair) look(e);
      const float w0 = v[i].x * down[0], w1 = v[i].y * down[1];
      const __half2 p = __floats2half2_rn(w0, w1);
      const float2 f = __half22float2(p);
      unsigned char* at = smem + T::RING + (e / (R / 2)) * T::H_PITCH + 4 * (e % (R / 2));
      *reinterpret_cast<uint32_t*>(at) = h2_as_u32(p);
      // (an infinity leaves any finite rest: fmaxf takes the number beside a NaN)
      *reinterpret_cast<uint32_t*>(at + T::H_BYTES) = h2_as_u32(__floats2half2_rn(fmaxf(w0 - f.x, -8.f), fmaxf(w1 - f.y, -8.f)));
    }
    __syncthreads();
    float acc[WT][CW / 8][4];
#pragma unroll
    for (int m = 0; m < WT; ++m)
#pragma unroll
      for (int i = 0; i < CW / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[m][i][k] = 0.f;
#pragma unroll
    for (int k = 0; k < kChunk / 16; ++k) {
      // columns: tokens 0-7, 8-15 of the step at columns 0-7, then at 8-15
      uint32_t xf[CW / 16][4];
#pragma unroll
      for (int i = 0; i < CW / 16; ++i)
        ldmatrix4_trans(xf[i], st + (16 * k + lane % 16) * T::X_PITCH + 2 * (CW * warp + 16 * i) + 16 * (lane / 16));
#pragma unroll
      for (int part = 1; part >= 0; --part)
#pragma unroll
        for (int m = 0; m < WT; ++m) {
          // ranks 0-7, 8-15 at tokens 0-7, then at 8-15
          uint32_t af[4];
          ldmatrix4_trans(af, parts + part * T::H_BYTES + (16 * k + 8 * (lane / 16) + lane % 8) * T::H_PITCH + 2 * rank0 +
                                  32 * m + 16 * (lane / 8 % 2));
#pragma unroll
          for (int i = 0; i < CW / 8; ++i) {
            const uint32_t bf[2] = {xf[i / 2][2 * (i % 2)], xf[i / 2][2 * (i % 2) + 1]};
            mma_16816(acc[m][i], af, bf);
          }
        }
    }
#pragma unroll
    for (int m = 0; m < WT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = rank0 + 16 * m + 8 * h + g;
        const float back = j < R ? __uint_as_float((uint32_t)(127 + exponent_of(top[j])) << 23) : 0.f;
#pragma unroll
        for (int i = 0; i < CW / 8; ++i) {
          total[m][i][2 * h] = fmaf(back, acc[m][i][2 * h], total[m][i][2 * h]);
          total[m][i][2 * h + 1] = fmaf(back, acc[m][i][2 * h + 1], total[m][i][2 * h + 1]);
        }
      }
  }
  cp_async_wait<0>();
  __syncthreads();                       // the ring is free
#pragma unroll
  for (int m = 0; m < WT; ++m)
#pragma unroll
    for (int i = 0; i < CW / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = rank0 + 16 * m + g + 8 * (k >> 1), c = CW * warp + 8 * i + 2 * t + (k & 1);
        if (j < R) sums[BY_ROWS ? c * PITCH + j : j * PITCH + c] = total[m][i][k];
      }
  cg::cluster_group cluster = cg::this_cluster();
  if (Z > 1) cluster.sync();
  else __syncthreads();
  const float f = a.scale ? ld_f32(a.scale + adapter) : 1.f;
  // rows of the output, four values a thread; the CTAs of a cluster take turns
  for (int e = threadIdx.x + z * kThreads; e < W * R / 4; e += Z * kThreads) {
    const int row = BY_ROWS ? e / (R / 4) : e / (W / 4), x4 = BY_ROWS ? e % (R / 4) : e % (W / 4);
    if ((BY_ROWS ? base + row : base + 4 * x4) >= a.C) continue;
    float4* at = reinterpret_cast<float4*>(BY_ROWS ? dst + (size_t)(base + row) * R + 4 * x4
                                                   : dst + (size_t)row * a.C + base + 4 * x4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < Z; ++k) {
      const float* from = Z > 1 ? cluster.map_shared_rank(sums, k) : sums;
      const float4 o = *reinterpret_cast<const float4*>(from + row * PITCH + 4 * x4);
      v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
    }
    v = make_float4(f * v.x, f * v.y, f * v.z, f * v.w);
    if (accumulate) {
      const float4 o = *at;
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *at = v;
  }
  if (Z > 1) cluster.sync();             // no CTA leaves while another reads its sums
}

template <int RJ>
__global__ void __launch_bounds__(kThreads, RJ <= 2 ? 3 : 2)
q4gsw_adapters_grad_kernel(const GradSide da, const GradSide db, const int32_t* plan, int M, int L, int groups_a,
                           int accumulate) {
  extern __shared__ __align__(16) unsigned char grad_smem[];
  __shared__ unsigned int s_top[2 * 8 * RJ];     // of this chunk and the next
  griddep_launch_dependents();
  griddep_wait();
  const PlanView P = plan_view(const_cast<int32_t*>(plan), M, L);
  if (!plan_fits(P, M, L)) return;
  if ((int)blockIdx.x < groups_a) grad_block<false, RJ>(da, P, blockIdx.x, accumulate, grad_smem, s_top);
  else grad_block<true, RJ>(db, P, blockIdx.x - groups_a, accumulate, grad_smem, s_top);
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
static cudaError_t down_form(cudaLaunchConfig_t& cfg, const __half* a, const __half* p, const float* scale,
                             const AdaptersRef& ad, float* out, int M, int C) {
  using D = ma::DownRing<BY_ROWS, RJ>;
  auto kernel = ma::q4gsw_adapters_down_kernel<BY_ROWS, RJ>;
  static PerDeviceOnce once;
  const cudaError_t e = once_per_device(once, current_device(), [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, D::BYTES);
  });
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = D::BYTES;
  unsigned int* error = nullptr;
  const cudaError_t w = device_error_word(&error);
  if (w != cudaSuccess) return w;
  return cudaLaunchKernelEx(&cfg, kernel, a, p, scale, ad.plan, out, M, ad.L, C, error);
}

cudaError_t launch_adapters_down(const AdaptersRef& ad, const uint16_t* act, bool by_rows, const uint16_t* proj,
                                 const float* scale, int M, int C, float* out, cudaStream_t stream) {
  const int groups = ma::plan_pairs(M, ad.L), sms = sm_count(current_device());
  // contraction splits: about two CTAs per SM, two stages each at least, clusters of at most
  // 8, by the pairs that are likely to be in use, half of the adapters' last ones (by all
  // that may be: 1024 tokens over 64 adapters 23.3 us, 17.9 now; 256 over 6 of them 11.9 and 8.5)
  const int last = ad.L + 1 < M / 16 ? ad.L + 1 : M / 16;
  const int likely = M / 32 + last / 2 < groups ? M / 32 + last / 2 : groups;
  const int stages = (C + 127) / 128;
  int KS = 1;
  while (KS < 8 && 2 * likely * KS <= 2 * sms && stages / (2 * KS) >= 2) KS *= 2;
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
#define Q4_DOWN(RJ_)                                                            \
  return by_rows ? down_form<true, RJ_>(cfg, a, p, scale, ad, out, M, C)        \
                 : down_form<false, RJ_>(cfg, a, p, scale, ad, out, M, C)
  Q4_RANKS(ad.r / 8, Q4_DOWN)
#undef Q4_DOWN
}

template <bool BY_ROWS, int RJ>
static cudaError_t up_form(cudaLaunchConfig_t& cfg, const float* inter, const __half* p, const float* scale,
                           const AdaptersRef& ad, const __half* res, __half* out, int M, int C, int per) {
  using U = ma::UpRing<BY_ROWS, RJ>;
  auto kernel = ma::q4gsw_adapters_up_kernel<BY_ROWS, RJ>;
  static PerDeviceOnce once;
  const cudaError_t e = once_per_device(once, current_device(), [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, U::BYTES_RES);
  });
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = res ? U::BYTES_RES : U::BYTES;
  return cudaLaunchKernelEx(&cfg, kernel, inter, p, scale, ad.plan, res, out, M, ad.L, C, per);
}

cudaError_t launch_adapters_up(const AdaptersRef& ad, const float* inter, bool by_rows, const uint16_t* proj,
                               const float* scale, int M, int C, const uint16_t* res, uint16_t* out,
                               cudaStream_t stream) {
  const int groups = (ma::plan_pairs(M, ad.L) + 1) / 2;
  const int blocks = (C + 63) / 64;
  // runs of two blocks or more: up to 16 CTAs per SM, so that those without an adapter
  // leave room (4096 x 14336, rank 64: 49.5 us, 51.3 with eight, 55.8 with four; 1021 x
  // 4096: 8.8 with single blocks, 7.3 with two)
  int runs = 16 * sm_count(current_device()) / groups;
  runs = runs < 1 ? 1 : runs > (blocks + 1) / 2 ? (blocks + 1) / 2 : runs;
  const int per = (blocks + runs - 1) / runs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(groups, (blocks + per - 1) / per, 1);
  cfg.blockDim = dim3(ma::kUpThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  serialize(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const __half* p = reinterpret_cast<const __half*>(proj);
  const __half* rs = reinterpret_cast<const __half*>(res);
  __half* o = reinterpret_cast<__half*>(out);
#define Q4_UP(RJ_)                                                              \
  return by_rows ? up_form<true, RJ_>(cfg, inter, p, scale, ad, rs, o, M, C, per)  \
                 : up_form<false, RJ_>(cfg, inter, p, scale, ad, rs, o, M, C, per)
  Q4_RANKS(ad.r / 8, Q4_UP)
#undef Q4_UP
}

template <bool FWD, int RJ, int U, int W>
static cudaError_t low_form(cudaLaunchConfig_t& cfg, int KS, const __half* act, const __half* down, const __half* up,
                            const float* scale, const AdaptersRef& ad, float* inter, const __half* res, __half* out,
                            int M, int C_down, int C_up) {
  constexpr int kTile = (int)sizeof(float) * ma::kTileRows * 8 * RJ;
  auto kernel = ma::q4gsw_adapters_low_kernel<FWD, RJ, U, W>;
  static PerDeviceOnce once;
  const cudaError_t e = once_per_device(once, current_device(), [&] {
    if (W == 4) {      // runs beside the product's CTAs: with their division of shared memory
      const cudaError_t c =
          cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
      if (c != cudaSuccess) return c;
    }
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (W + 8) * kTile);
  });
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = (W + (KS > 1 ? KS : 0)) * kTile;
  cfg.blockDim = dim3(32 * W, 1, 1);
  unsigned int* error = nullptr;
  const cudaError_t w = device_error_word(&error);
  if (w != cudaSuccess) return w;
  return cudaLaunchKernelEx(&cfg, kernel, act, down, up, scale, ad.plan, inter, res, out, M, ad.L, C_down, C_up, error);
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
  // The forward product of 9 to 16 tokens has two CTAs of 288 threads on every SM at once,
  // and one that starts late ends late.  CTAs of four warps with 80 registers a thread leave
  // them room (10240 of 65536) and run beside them, where the product is long enough for
  // their own pace: 16 tokens on 4096 x 14336 22.5 -> 18.1 us, on 14336 x 4096 23.2 -> 18.8
  // (9 tokens 17.6 -> 18.4), on 4096 x 4096 13.3 -> 11.0; but on 8192 x 2048 14.1 -> 15.5.
  // (Backward: 30.7 -> 25.6, 29.4 -> 31.6, 17.0 -> 19.3 and 20.7 -> 17.0: eight warps.)
  const bool beside = fwd && M > 8 && M <= 16 && (long long)N * K >= 2048LL * (N + K);
  // Up to 8 tokens the product's CTAs are smaller and leave a few places free: four warps
  // with two chunks in flight, where `down` is at least as long as `up` (4 and 6 tokens on
  // 4096 x 14336 17.8 -> 14.3 and 18.3 -> 14.8, on 4096 x 4096 9.4 -> 9.4 and 11.9 -> 9.7; but
  // on 8192 x 2048 10.5 -> 11.2 and 12.7 -> 11.4, on 14336 x 4096 15.4 -> 16.0 and 15.5 -> 16.4).
  const bool slim = fwd && M <= 8 && K >= N;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(slots, KS, 1);
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
    if constexpr (RJ_ <= 2) {                                                                                         \
      if (beside) return low_form<true, RJ_, 1, 4>(cfg, KS, x, pa, pb, scale, ad, inter, rs, o, M, K, N);             \
      if (slim) return low_form<true, RJ_, 2, 4>(cfg, KS, x, pa, pb, scale, ad, inter, rs, o, M, K, N);               \
    }                                                                                                                 \
    return fwd ? (deep ? low_form<true, RJ_, U, 8>(cfg, KS, x, pa, pb, scale, ad, inter, rs, o, M, K, N)              \
                       : low_form<true, RJ_, 1, 8>(cfg, KS, x, pa, pb, scale, ad, inter, rs, o, M, K, N))             \
               : (deep ? low_form<false, RJ_, U, 8>(cfg, KS, x, pb, pa, scale, ad, inter, rs, o, M, N, K)             \
                       : low_form<false, RJ_, 1, 8>(cfg, KS, x, pb, pa, scale, ad, inter, rs, o, M, N, K));           \
  }
  Q4_RANKS(ad.r / 8, Q4_LOW)
#undef Q4_LOW
}

template <int RJ>
static cudaError_t grad_form(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, const AdaptersRef& ad,
                             const ma::GradSide& da, const ma::GradSide& db, int M, bool accumulate) {
  using T = ma::GradTile<RJ>;
  auto kernel = ma::q4gsw_adapters_grad_kernel<RJ>;
  static PerDeviceOnce once;
  const cudaError_t e = once_per_device(once, current_device(), [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::BYTES);
  });
  if (e != cudaSuccess) return e;
  const int ga = (da.C + T::W - 1) / T::W, gb = (db.C + T::W - 1) / T::W;
  // token splits: about two CTAs per SM, two chunks each where the adapters have equal shares
  int Z = 1;
  while (Z < 8 && (long long)(ga + gb) * ad.L * Z < 2LL * sm_count(current_device()) &&
         M / ad.L >= 4 * Z * ma::kChunk)
    Z *= 2;
  cfg.gridDim = dim3(ga + gb, ad.L, Z);
  cfg.blockDim = dim3(ma::kThreads, 1, 1);
  cfg.dynamicSmemBytes = T::BYTES;
  attr->val.clusterDim.z = Z;
  return cudaLaunchKernelEx(&cfg, kernel, da, db, ad.plan, M, ad.L, ga, (int)accumulate);
}

cudaError_t launch_adapters_grad(const AdaptersRef& ad, const uint16_t* x, const float* v, float* d_a, int K,
                                 const uint16_t* d_y, const float* u, const float* scale, float* d_b, int N, int M,
                                 bool accumulate, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  serialize(attr[0]);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const ma::GradSide da{reinterpret_cast<const __half*>(x), v, nullptr, d_a, K};
  const ma::GradSide db{reinterpret_cast<const __half*>(d_y), u, scale, d_b, N};
#define Q4_GRAD(RJ_) return grad_form<RJ_>(cfg, &attr[1], ad, da, db, M, accumulate)
  Q4_RANKS(ad.r / 8, Q4_GRAD)
#undef Q4_GRAD
}

}  // namespace q4gsw
