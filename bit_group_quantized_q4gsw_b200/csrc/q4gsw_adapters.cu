// q4gsw_adapters.cu - the low-rank half of a projection with an adapter for
// every token, and the gradients of the adapters (sm_100a).
//
// Over the tiles of a plan (16 tokens of one adapter each):
//   down   u = x A^T (forward), v = s d_y B (backward): the intermediate, fp32 [M][r]
//   few    the same for few tiles
//   grad   d_A = v^T x, d_B = s d_y^T u over the tokens of each adapter, fp32
// The base product adds s u B^T (or v A) to its own sums while they are fp32
// (q4gsw_lowrank.cuh), on its routes at any number of tokens and with either kind of
// scales.  The first kernel lets the next start only behind its own wait; the product,
// launched behind it, then knows its activations to be complete, reads them at once and
// waits for the intermediate in its epilogue alone.
//
// The intermediate stays in fp32: rounded to fp16 it would put 2^-11 of error into
// fp32 gradients, and small gradients would fall below fp16's range.  It goes to the
// tensor cores as two fp16 parts over a power of two near the largest value of the
// token's row (in the product) or of the rank's chunk of tokens (`grad`): 2^-23 of that
// is lost.
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
// is given) of the tile's adapter, for many tiles (few: q4gsw_adapters_few_kernel).
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

// ---------------------------------------------------------------- few
// The same for few tiles: a cluster of KS CTAs has one tile, and its CTAs split the
// contraction.  Each gets the sums of all of them for its share of the tile's rows (every
// CTA writes to every other's shared memory, added in rank order).
//
// W warps: eight, or four beside the product of up to 16 tokens (launch_adapters_few).
// The registers are kept to three CTAs an SM where a warp has one chunk and the rank is at
// most 16: with the columns of x forward that spills (100 bytes a thread of stores with rank
// 8, 40 with 16) and is still the faster where the tiles are many (three, two, one CTA an SM,
// us of a whole call on 8192 x 2048, rank 8: 48 tokens of as many adapters 22.9, 24.0, 27.0;
// 256 tokens of 31 27.6, 28.3, 30.4; 256 of 8 24.7, 24.3, 25.2; 32 of 8 16.1, 16.0, 15.9).
template <bool BY_ROWS, int RJ, int U, int W>
__global__ void __launch_bounds__(32 * W, W == 4 ? 4 : U == 1 && RJ <= 2 ? 3 : 1)
q4gsw_adapters_few_kernel(const __half* act, const __half* proj, const float* scale, const int32_t* plan, float* out,
                          int M, int L, int C, unsigned int* error) {
  constexpr int R = 8 * RJ;
  extern __shared__ __align__(16) float few_smem[];
  auto red = reinterpret_cast<float (*)[kTileRows][R]>(few_smem);                       // [W]
  auto recv = reinterpret_cast<float (*)[R]>(few_smem + W * kTileRows * R);             // [KS][owned rows], by sender
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
  if (adapter < 0) {               // the whole cluster
    for (int e = threadIdx.x + 32 * W * ks; e < kTileRows * R; e += 32 * W * KS) {
      const int to = ld_int(rows + e / R);
      if (to >= 0) out[(size_t)to * R + e % R] = 0.f;
    }
    return;
  }
  if (KS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int r0 = ld_int(rows);
  const __half* a0 = act + (size_t)(m[0] < 0 ? r0 : m[0]) * C;
  const __half* a1 = act + (size_t)(m[1] < 0 ? r0 : m[1]) * C;
  const int chunks = (C + 63) / 64, parts = KS * W, part = ks * W + warp;
  const int s_begin = (int)((long long)part * chunks / parts), s_end = (int)((long long)(part + 1) * chunks / parts);
  float acc[RJ][4];
#pragma unroll
  for (int j = 0; j < RJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  down_chunks<BY_ROWS, RJ, U>(proj + (size_t)adapter * R * C, a0, a1, C, s_begin, s_end, g, t, acc);
  down_park<BY_ROWS, RJ>(acc, red[warp], g, t);
  __syncthreads();
  auto own = [&](int row, int j) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[w][row][j];
    return s;
  };
  const int owned = kTileRows / KS;      // rows that this CTA writes (KS is a power of two)
  if (KS > 1) {
    // every CTA of the cluster has started (arrived above): remote stores are safe
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    for (int e = threadIdx.x; e < kTileRows * R; e += 32 * W) {
      const int row = e / R, j = e % R;
      *cluster.map_shared_rank(&recv[ks * owned + row % owned][j], row / owned) = own(row, j);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  for (int e = threadIdx.x; e < owned * R; e += 32 * W) {
    const int row = e / R, j = e % R, to = ld_int(rows + ks * owned + row);
    if (to < 0) continue;
    float v = 0.f;
    if (KS > 1) {
      for (int q = 0; q < KS; ++q) v += recv[q * owned + row][j];
    } else {
      v = own(row, j);
    }
    out[(size_t)to * R + j] = scale ? ld_f32(scale + adapter) * v : v;
  }
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
// range, and the tensor cores' own sums are four products long (two steps of tokens of both
// parts).  The Z CTAs of a cluster take every Z-th chunk, and their sums are added through
// distributed shared memory in rank order.
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

// Up to 256 tokens in at most 48 tiles.  On both sides (us of a whole call, few and down): 128
// tokens of one adapter of 32, 4096 x 14336, rank 64 36.3 and 44.5, 256 46.6 and 49.7, 8192 x
// 2048, rank 16 25.3 and 24.8; 512 tokens of eight adapters there 28.9 and 28.5, backward 35.6
// and 33.1, 700 tokens 53.6 and 50.1; 96 tokens of as many adapters on 4096 x 14336, rank 64
// 115 and 86, 48 75.6 and 62.1, 16 of 32 26.3 and 31.8.
bool adapters_few(const AdaptersRef& ad, int M) { return M <= 256 && ma::plan_slots(M, ad.L) <= 48; }

template <bool BY_ROWS, int RJ, int U, int W>
static cudaError_t few_form(cudaLaunchConfig_t& cfg, const __half* act, const __half* proj, const float* scale,
                            const AdaptersRef& ad, float* out, int M, int C) {
  constexpr int kTile = (int)sizeof(float) * ma::kTileRows * 8 * RJ;
  constexpr int kBytes = (W + 1) * kTile;      // the warps' sums, and those that the cluster sends
  auto kernel = ma::q4gsw_adapters_few_kernel<BY_ROWS, RJ, U, W>;
  static PerDeviceOnce once;
  const cudaError_t e = once_per_device(once, current_device(), [&] {
    if (W == 4) {      // runs beside the product's CTAs: with their division of shared memory
      const cudaError_t c =
          cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
      if (c != cudaSuccess) return c;
    }
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  });
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = kBytes;
  cfg.blockDim = dim3(32 * W, 1, 1);
  unsigned int* error = nullptr;
  const cudaError_t w = device_error_word(&error);
  if (w != cudaSuccess) return w;
  return cudaLaunchKernelEx(&cfg, kernel, act, proj, scale, ad.plan, out, M, ad.L, C, error);
}

static cudaError_t launch_adapters_few(const AdaptersRef& ad, const __half* x, bool by_rows, const __half* p,
                                       const float* scale, int M, int C, float* out, cudaStream_t stream) {
  const int KS = 8;
  const bool deep = (C + 63) / 64 > KS * ma::kWarps;      // more than a chunk a warp
  // The forward product of up to 16 tokens has two or four CTAs on every SM at once, and one
  // that starts late ends late.  CTAs of four warps leave them room and run beside them
  // (four and eight warps, us of a whole call, rank 16): 16 tokens of as many adapters on 4096
  // x 14336 17.7 and 20.4, on 8192 x 2048 11.2 and 13.2; of one adapter 17.3 and 17.7, 10.8 and
  // 10.9; 8 tokens 16.3 and 15.7, 9.7 and 10.5.
  const bool slim = by_rows && M <= ma::kTileRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ma::plan_slots(M, ad.L), KS, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  serialize(attr[0]);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = KS;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
#define Q4_FEW(RJ_)                                                                              \
  {                                                                                              \
    constexpr int U = RJ_ <= 2 ? 4 : RJ_ <= 4 ? 2 : 1;                                           \
    if constexpr (RJ_ <= 2) {                                                                    \
      if (slim) return few_form<true, RJ_, 2, 4>(cfg, x, p, scale, ad, out, M, C);               \
    }                                                                                            \
    return by_rows ? (deep ? few_form<true, RJ_, U, 8>(cfg, x, p, scale, ad, out, M, C)          \
                           : few_form<true, RJ_, 1, 8>(cfg, x, p, scale, ad, out, M, C))         \
                   : (deep ? few_form<false, RJ_, U, 8>(cfg, x, p, scale, ad, out, M, C)         \
                           : few_form<false, RJ_, 1, 8>(cfg, x, p, scale, ad, out, M, C));       \
  }
  Q4_RANKS(ad.r / 8, Q4_FEW)
#undef Q4_FEW
}

cudaError_t launch_adapters_down(const AdaptersRef& ad, const uint16_t* act, bool by_rows, const uint16_t* proj,
                                 const float* scale, int M, int C, float* out, cudaStream_t stream) {
  const __half* a = reinterpret_cast<const __half*>(act);
  const __half* p = reinterpret_cast<const __half*>(proj);
  if (adapters_few(ad, M)) return launch_adapters_few(ad, a, by_rows, p, scale, M, C, out, stream);
  const int groups = ma::plan_pairs(M, ad.L), sms = sm_count(current_device());
  // Contraction splits: two stages each at least, clusters of at most 8.  The pairs in use
  // are at least M / 32 and at most `groups`, which of the two the host does not know: no
  // more than two CTAs per SM by the least and four by the most.  Calls with 1, 2, 4, 8 splits (us,
  // the choice in brackets), rank 64, 4096 x 4096: 128 tokens of as many adapters 67.7, 56.4,
  // [54.1], 66.2, 256 of as many 77.9, [82.8], 92.6, 113, 256 of six of 64 adapters 41.0, 39.0,
  // 32.3, [29.4], 1024 of 64 84.5, 74.6, [68.8], 75.5, 4096 of 16 191, [177], 184, 194.
  const int stages = (C + 127) / 128;
  int KS = 1;
  while (KS < 8 && 2LL * KS * groups <= 4 * sms && 2LL * KS * (M / 32) <= 2 * sms && stages / (2 * KS) >= 2) KS *= 2;
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
#define Q4_DOWN(RJ_)                                                            \
  return by_rows ? down_form<true, RJ_>(cfg, a, p, scale, ad, out, M, C)        \
                 : down_form<false, RJ_>(cfg, a, p, scale, ad, out, M, C)
  Q4_RANKS(ad.r / 8, Q4_DOWN)
#undef Q4_DOWN
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
