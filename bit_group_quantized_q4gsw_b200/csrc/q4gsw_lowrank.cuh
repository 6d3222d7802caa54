// q4gsw_lowrank.cuh - the low-rank term of a projection with an adapter for every
// token, in the epilogue of its base product (sm_100a).
//
//   y[m][c] = fp16(sums[m][c] + s_a sum_j inter[m][j] P_a(c, j) + bias[c] + res[m][c])
//
// with a the token's adapter, P_a(c, j) = mat[a][c][j] (forward: B [L, N, r]) or
// mat[a][j][c] (backward: A [L, r, K]).  The term is added to the product's sums while
// these are fp32, so that y is rounded once: a term that passes fp16's range and is brought
// back by the base product gives what the formula says, and none of its bits are lost
// where the two cancel.  (As fp16 in the output's place, between a kernel of its own
// and the product, it cost half a unit in the last place of itself, and was infinite
// from 65520 on.)
//
// Up to 16 tokens (GEMV) a thread has two columns of a token and adds r products for
// each, in fp32 (finish_pair).  Above, the term of the tokens of a tile that have one adapter
// goes through the tensor cores (add_terms).
#pragma once

#include "q4gsw_adapters.cuh"
#include "q4gsw_epilogue.cuh"
#include "q4gsw_sm100.cuh"

namespace q4gsw {
namespace lr {

using ma::PlanView;
using ma::plan_view;

// Coherent loads, as in q4gsw_adapters.cu.
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
__device__ __forceinline__ int ld_int(const int32_t* p) { return (int)ld_u32(p); }

// Whether the plan is the call's (the kernel in front has recorded that it is not).
__device__ __forceinline__ bool plan_fits(const EpiLow& o) {
  const uint4 h = ld_v4(o.plan);
  return (int)h.y == o.M && (int)h.z == o.L && (int)h.w == ma::kPlanMark;
}

// ---------------------------------------------------------------- up to 16 tokens
// The adapters of tokens 0 .. 15 (-1: none; -2: the plan is not the call's, and nothing is
// written), by one warp, before griddepcontrol.wait: the plan was complete before the
// kernel in front could start, as the activations were.
__device__ __forceinline__ void few_adapters(const EpiLow& o, int16_t* adapter) {
  const int lane = threadIdx.x & 31;
  const int head = (int)ld_l2_u32(o.plan + 1 + lane % 3);
  const bool fits = __all_sync(0xffffffffu, head == (lane % 3 == 0 ? o.M : lane % 3 == 1 ? o.L : ma::kPlanMark));
  if (lane < 16) adapter[lane] = fits ? -1 : -2;
  __syncwarp();
  if (fits) {
    const PlanView P = plan_view(const_cast<int32_t*>(o.plan), o.M, o.L);
    const int n = ma::kTileRows * ma::plan_slots(o.M, o.L);
#pragma unroll 4
    for (int i = lane; i < n; i += 32) {
      const int m = (int)ld_l2_u32(P.rows + i), a = (int)ld_l2_u32(P.tile + i / ma::kTileRows);
      if (m >= 0) adapter[m] = (int16_t)(a >= 0 ? a : -1);
    }
  }
  __syncwarp();
}

// What tokens [tb, te) need of the matrix for columns [c0, c0 + cols) on its way to L2, by one warp.
template <bool BY_ROWS>
__device__ __forceinline__ void few_prefetch(const EpiLow& o, const int16_t* adapter, int tb, int te, int c0, int cols) {
  const int lane = threadIdx.x & 31;
  for (int m = tb; m < te; ++m) {
    const int a = adapter[m];
    if (a < 0) continue;
    const __half* p = o.mat + (size_t)a * o.r * o.N;
    if (BY_ROWS) {
      for (int e = 64 * lane; e < cols * o.r; e += 64 * 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p + (size_t)c0 * o.r + e));
    } else {
      for (int e = lane; e < 2 * o.r; e += 32)
        if (64 * (e & 1) < cols) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + (size_t)(e >> 1) * o.N + c0 + 64 * (e & 1)));
    }
  }
}

// Columns c, c + 1 (c even; N % 8 == 0: both or neither are there) of token m with adapter
// a (few_adapters), whose sums are v.  What is read is on its way before the first use.
template <bool BY_ROWS>
__device__ __forceinline__ void finish_pair(const EpiLow& o, int a, int m, int c, float2 v) {
  if (a < -1) return;
  const size_t at = (size_t)m * o.N + c;
  const uint32_t bias = o.bias ? ld_u32(o.bias + c) : 0u, res = o.res ? ld_u32(o.res + at) : 0u;
  if (a >= 0) {
    const float f = o.scale ? __uint_as_float(ld_u32(o.scale + a)) : 1.f;
    const float* u = o.inter + (size_t)m * o.r;
    float t0 = 0.f, t1 = 0.f;
    if (BY_ROWS) {
      const __half* p = o.mat + ((size_t)a * o.N + c) * o.r;
#pragma unroll 2
      for (int j = 0; j < o.r; j += 8) {                          // r % 8 == 0
        const uint4 w0 = ld_v4(p + j), w1 = ld_v4(p + o.r + j), q0 = ld_v4(u + j), q1 = ld_v4(u + j + 4);
        const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w},
                       q[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 p0 = __half22float2(u32_as_h2(a0[e])), p1 = __half22float2(u32_as_h2(a1[e]));
          t0 = fmaf(__uint_as_float(q[2 * e]), p0.x, t0);
          t1 = fmaf(__uint_as_float(q[2 * e]), p1.x, t1);
          t0 = fmaf(__uint_as_float(q[2 * e + 1]), p0.y, t0);
          t1 = fmaf(__uint_as_float(q[2 * e + 1]), p1.y, t1);
        }
      }
    } else {
      const __half* p = o.mat + (size_t)a * o.r * o.N + c;
      for (int j = 0; j < o.r; j += 8) {
        const uint4 q0 = ld_v4(u + j), q1 = ld_v4(u + j + 4);
        const uint32_t q[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = ld_u32(p + (size_t)(j + e) * o.N);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 k = __half22float2(u32_as_h2(w[e]));
          t0 = fmaf(__uint_as_float(q[e]), k.x, t0);
          t1 = fmaf(__uint_as_float(q[e]), k.y, t1);
        }
      }
    }
    v.x = fmaf(f, t0, v.x);
    v.y = fmaf(f, t1, v.y);
  }
  const float2 b = __half22float2(u32_as_h2(bias)), r = __half22float2(u32_as_h2(res));
  *reinterpret_cast<uint32_t*>(o.y + at) = h2_as_u32(__floats2half2_rn(v.x + b.x + r.x, v.y + b.y + r.y));
}

// ---------------------------------------------------------------- tiles
// A GEMM with this epilogue has two more warps than without.  While the others are in
// the main loop they find which tokens of the CTA's output have which adapter (find); the
// epilogue then adds the term to the parked sums of up to 128 or 256 tokens at a time
// (add_terms).
constexpr int kFindWarps = 2;
constexpr int kChunk = 128;
// Two lists of tokens with an adapter, those of one side by side.
struct Groups {
  int count[2];                        // tokens
  int fits;                            // the plan is the call's
  float factor[2][kChunk];
  int16_t adapter[2][kChunk];
  unsigned char row[2][kChunk];        // from the first token of the list's range on
};
struct Ranges {
  int begin[2], end[2];                // tokens, at most 128 each
};
// Shared memory beside the parked sums: inter of one list's tokens, or up to rank 32 of both,
// as fp32 [r], then as two fp16 parts over 2^k, hi and lo, of 32 or 64 ranks each (zeros from
// r on).  A row has an odd number of 16 bytes.
__device__ __forceinline__ bool both_lists(int r) { return r <= 32; }
__device__ __forceinline__ int part_bytes(int r) { return both_lists(r) ? 64 : 128; }
__device__ __forceinline__ int pitch_of(int r) { return 2 * part_bytes(r) + 16; }
constexpr int kZeroBytes = 2 * 128 + 16;
struct Scratch {
  unsigned char inter[2 * kChunk * (2 * 64 + 16)];
  unsigned char zeros[kZeroBytes];                   // a row of a token that is not there
  float back[2 * kChunk];                            // 2^k
};
static_assert(sizeof(Scratch::inter) >= kChunk * (2 * 128 + 16) && sizeof(Scratch::inter) % 16 == 0, "either layout");

// Has the rows' inter copied to shared memory, by `threads` threads, for add_terms.
__device__ __forceinline__ void stage(const EpiLow& o, Scratch* s, int m0, int rows, int tid, int threads) {
  const int vectors = o.r / 4, pitch = pitch_of(o.r);
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(s->inter);
#pragma unroll 1
  for (int e = tid; e < rows * vectors; e += threads) {
    const int row = e / vectors, x = e - row * vectors;
    cp_async_16(to + row * pitch + 16 * x, o.inter + (size_t)(m0 + row) * o.r + 4 * x);
  }
  cp_async_commit();
}

// The exponent k of a float's pattern (2^k <= |v| < 2^(k + 1)), held where 2^k and 2^-k
// are both normal numbers.
__device__ __forceinline__ int exponent_of(uint32_t bits) { return max(-126, min((int)(bits >> 23 & 255u) - 127, 126)); }
__device__ __forceinline__ float power_of_two(int k) { return __uint_as_float((uint32_t)(127 + k) << 23); }
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

// The lists of both ranges, by the threads `tid` = 0 .. 63 (whole warps) of a CTA that has
// set count and fits to zero behind a barrier.  A plan's order has the tokens of an
// adapter in their own order, so those of a range stand side by side: `lanes` lanes search
// the ends of that run, each step narrows it lanes + 1 times, two adapters at once.
// Which adapter stands where depends on the order of atomics, the results do not: every
// value of the output is one adapter's.
__device__ __forceinline__ void find(const EpiLow& o, Groups* s, const Ranges& range, int tid) {
  constexpr int kSearch = 32 * kFindWarps, A = 2;
  griddep_wait();
  if (!plan_fits(o)) return;
  if (tid == 0) s->fits = 1;
  const PlanView P = plan_view(const_cast<int32_t*>(o.plan), o.M, o.L);
  int lanes = 32;
  while (lanes > 1 && o.L * lanes > kSearch) lanes >>= 1;
  const int lane = tid & 31, sub = lane & (lanes - 1), step = kSearch / lanes;
  const uint32_t mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (lane - sub);
  const int key[4] = {range.begin[0], range.end[0], range.begin[1], range.end[1]};
  for (int a0 = tid / lanes; __any_sync(0xffffffffu, a0 < o.L); a0 += A * step) {
    int lo[A][4], n[A][4], any = 0;
#pragma unroll
    for (int i = 0; i < A; ++i) {
      const int a = a0 + i * step;
      const int b = a < o.L ? ld_int(P.first + a) : 0, e = a < o.L ? ld_int(P.first + a + 1) : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) lo[i][k] = b, n[i][k] = e - b;
      any |= e - b;
    }
    while (__any_sync(0xffffffffu, any)) {
      any = 0;
      int token[A][4];
#pragma unroll
      for (int i = 0; i < A; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = (n[i][k] + lanes) / (lanes + 1) * (sub + 1) - 1;      // n > 0: at >= 0
          token[i][k] = n[i][k] > 0 && at < n[i][k] ? ld_int(P.order + lo[i][k] + at) : 0x7fffffff;
        }
#pragma unroll
      for (int i = 0; i < A; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int w = (n[i][k] + lanes) / (lanes + 1);
          const int c = __popc(__ballot_sync(0xffffffffu, token[i][k] < key[k]) & mask);
          const int left = n[i][k] - c * w;
          lo[i][k] += c * w;
          n[i][k] = max(0, c < lanes ? min(left, w - 1) : left);
          any |= n[i][k];
        }
    }
#pragma unroll
    for (int i = 0; i < A; ++i)
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        const int from = lo[i][2 * l], tokens = max(0, lo[i][2 * l + 1] - from), a = a0 + i * step;
        int place = 0;
        if (sub == 0 && tokens) place = atomicAdd(&s->count[l], tokens);
        place = __shfl_sync(0xffffffffu, place, lane - sub);
        const float f = o.scale && tokens ? __uint_as_float(ld_u32(o.scale + a)) : 1.f;
        for (int k = sub; k < tokens; k += 4 * lanes) {
          int token[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) token[e] = k + e * lanes < tokens ? ld_int(P.order + from + k + e * lanes) : 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k + e * lanes < tokens) {
              const int at = place + k + e * lanes;
              s->row[l][at] = (unsigned char)(token[e] - key[2 * l]);
              s->adapter[l][at] = (int16_t)a;
              s->factor[l][at] = f;
            }
        }
      }
  }
}

// The sum of four columns over the partial tiles of S CTAs in rank order, N loads in
// flight: part(k) reads rank k's.
template <int N, class Part>
__device__ __forceinline__ float4 add_parts(int S, Part&& part) {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k = 0; k < S; k += N) {
    float4 p[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (k + i < S) p[i] = part(k + i);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (k + i < S) acc = make_float4(acc.x + p[i].x, acc.y + p[i].y, acc.z + p[i].z, acc.w + p[i].w);
  }
  return acc;
}

// Adds the low-rank term of list `l` (and, where both_lists and `two`, of the next) to the sums
// of the `rows` tokens from the list's range on (the second range kChunk behind the first),
// columns c0 .. of COLS, in shared memory: at(row, column) is the address of four columns'
// sums, side by side.  All THREADS threads of the CTA, with a barrier between what they
// parked and this (and `stage` before that); one ends it.
//
// inter goes to the tensor cores as two fp16 parts over a power of two with the row's
// largest value in [1, 2): 2^-23 of that value is lost.  A warp has 16 columns and a share
// of the lists, 16 tokens at a time, whose rows lie anywhere in the chunk (ldmatrix takes each
// row's address).  For each adapter of the 16 the other tokens' rows are zeros, and the
// sums of its own rows alone are taken (an infinite matrix times zeros is none of the
// others' business).  Adapters that follow each other share the matrix's fragments, which
// come from L2 into registers.
//
// The order of the ranks in the contraction is free: lane t of a quad has the r / 4 ranks
// from t r / 4 on, four of them in each step, so that a row of B [N, r] comes in vectors.
// The order of the columns is, too: column n of the j-th eight is 2 n + j.  A lane then
// reads two columns of a row of A [r, K] at once, and has the sums of four columns side by
// side.
//
// 512 tokens of eight adapters, rank 16, 8192 x 2048: 4 us of a call's 30.5; 4096 tokens of 16,
// rank 64, 14336 x 4096: 100 of 515, of which the tensor cores' part is 60 (49 as a kernel of its
// own, and the output through memory once more).  Bound by issued instructions and short
// chains: cold code, a few loads, four warps a scheduler.  So it has no long unrolled loops
// and next to no spills (what the GEMM leaves of L1 does not hold them: 4 bytes a thread in the
// forward GEMM, 72 in the backward one, which has 24 without the term; twice as many columns a
// warp with 84 bytes of them 531 us); outputs written from here in pieces of 32 bytes a row took 518,
// the next adapter's matrix in registers ahead of its use 550.
// 1024 scattered tokens of 64 adapters, some 56 to a chunk, rank 16: 97 us on 8192 x 2048, 160 on
// 4096 x 14336, backward 93 and 330 (112, 175, 113, 392 with 16 rows for each adapter): an
// adapter's matrix is taken again for every chunk of 128 tokens.
template <bool BY_ROWS, int COLS, int THREADS, class At>
__device__ __forceinline__ void add_terms(const EpiLow& o, const Groups* q, int l, bool two, Scratch* s, int rows,
                                          int c0, const At& at) {
  constexpr int WARPS = THREADS / 32, BLOCKS = COLS / 16, SHARES = WARPS / BLOCKS, STEPS = 4;
  // (volatile: what follows from it is computed here, not kept in registers around the loop
  // over chunks)
  int tid;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
  const int warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int per = o.r / 4;                           // ranks of a lane
  const int block = warp % BLOCKS, share = warp / BLOCKS;
  const int base = c0 + 16 * block;
  // batches of 16 tokens, of the first list and of the second
  const int batches0 = (q->count[l] + 15) / 16, batches = batches0 + (two ? (q->count[1] + 15) / 16 : 0);
  const bool works = share < SHARES && base < o.N;
  const int begin = works ? share * batches / SHARES : 0, end = works ? (share + 1) * batches / SHARES : 0;
  uint32_t bf[STEPS][2][2];                          // the matrix: [step of 16 ranks][eight columns]
  int mine = -1;
  auto fetch = [&](int a) {
    mine = a;
    const __half* mat = o.mat + (size_t)a * o.r * o.N;
    const int c = base + 2 * g < o.N ? base + 2 * g : base;      // N % 8 == 0: both columns or none
    if (BY_ROWS) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __half* p = mat + (size_t)(c + j) * o.r + t * per;
        uint32_t w[2 * STEPS];
        if (per % 8 == 0) {                          // vectors of what the rank's alignment allows
#pragma unroll
          for (int i = 0; i < STEPS / 2; ++i) {
            const uint4 x = 8 * i < per ? *reinterpret_cast<const uint4*>(p + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
          }
        } else if (per % 4 == 0) {
#pragma unroll
          for (int i = 0; i < STEPS; ++i) {
            const uint2 x = 4 * i < per ? *reinterpret_cast<const uint2*>(p + 4 * i) : make_uint2(0u, 0u);
            w[2 * i] = x.x, w[2 * i + 1] = x.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2 * STEPS; ++i) w[i] = 2 * i < per ? *reinterpret_cast<const uint32_t*>(p + 2 * i) : 0u;
        }
#pragma unroll
        for (int k = 0; k < STEPS; ++k) bf[k][j][0] = w[2 * k], bf[k][j][1] = w[2 * k + 1];
      }
    } else {
      const __half* p = mat + (size_t)(t * per) * o.N + c;
      // ranks up to 32 and the rest, all on their way before the first is used
      const bool rest = per > 8;
      uint32_t w[2][8];
      auto load = [&](int x) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[x][e] = 8 * x + e < per ? *reinterpret_cast<const uint32_t*>(p + (size_t)(8 * x + e) * o.N) : 0u;
      };
      auto turn = [&](int x) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              bf[2 * x + k][j][e] = prmt(w[x][4 * k + 2 * e], w[x][4 * k + 2 * e + 1], j ? 0x7632u : 0x5410u);
      };
      load(0);
      if (rest) load(1);
      turn(0);
      if (rest) turn(1);
    }
  };
  if (tid < kZeroBytes / 4) reinterpret_cast<uint32_t*>(s->zeros)[tid] = 0u;
  cp_async_wait<0>();
  __syncthreads();
  if (batches == 0) return;
  if (begin < end) fetch(begin < batches0 ? q->adapter[l][16 * begin] : q->adapter[1][16 * (begin - batches0)]);
  // ranks 2 sub, 2 sub + 1 of a row in a thread, 8, 16 or 32 lanes to a row, which is replaced
  // by its parts: rank t per + e stands where step e / 4 has it, and behind the ranks zeros
  // fill the last step
  const int lanes = o.r <= 16 ? 8 : o.r <= 32 ? 16 : 32, sub = lane % lanes;
  const int e0 = 2 * sub % per, pitch = pitch_of(o.r), lo = part_bytes(o.r);
  const int pos = 2 * sub < o.r ? 16 * (e0 / 4) + 8 * (e0 / 2 % 2) + 2 * (2 * sub / per) : 2 * sub;
#pragma unroll 2
  for (int row0 = 32 * warp / lanes; row0 < rows; row0 += THREADS / lanes) {      // the warp's rows from here on
    const int row = row0 + lane / lanes;
    unsigned char* from = s->inter + row * pitch;
    uint2 v = make_uint2(0u, 0u);
    if (row < rows && 2 * sub < o.r) v = *reinterpret_cast<const uint2*>(from + 8 * sub);
    uint32_t top = max(v.x & 0x7fffffffu, v.y & 0x7fffffffu);
    if (lanes == 32) top = __reduce_max_sync(0xffffffffu, top);
    else
      for (int x = lanes / 2; x; x /= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
    __syncwarp();                                    // the row is in registers
    if (row >= rows) continue;
    const int k = exponent_of(top);                  // an infinite or NaN value stays what it is
    const float w0 = __uint_as_float(v.x) * power_of_two(-k), w1 = __uint_as_float(v.y) * power_of_two(-k);
    const __half2 hi = __floats2half2_rn(w0, w1);
    const float2 back = __half22float2(hi);
    *reinterpret_cast<uint32_t*>(from + 2 * pos) = h2_as_u32(hi);
    // (an infinity leaves no rest)
    *reinterpret_cast<uint32_t*>(from + lo + 2 * pos) =
        h2_as_u32(__floats2half2_rn(isinf(w0) ? 0.f : w0 - back.x, isinf(w1) ? 0.f : w1 - back.y));
    if (sub == 0) s->back[row] = power_of_two(k);
  }
  __syncthreads();
  const uint32_t parts = (uint32_t)__cvta_generic_to_shared(s->inter), zeros = (uint32_t)__cvta_generic_to_shared(s->zeros);
#pragma unroll 1
  for (int i = begin; i < end; ++i) {
    const int list = i < batches0 ? l : 1, p0 = 16 * (i < batches0 ? i : i - batches0), p = p0 + (lane & 15);
    const bool in = p < q->count[list];
    const int a_of = in ? q->adapter[list][p] : -1, row_of = in ? q->row[list][p] + (list - l) * kChunk : 0;
    const uint32_t from = parts + row_of * pitch + 16 * (lane >> 4);
    float sum[2][4];                                 // of eight columns each
    uint32_t todo = __ballot_sync(0xffffffffu, in) & 0xffffu;
#pragma unroll 1
    while (todo) {
      const int a = __shfl_sync(0xffffffffu, a_of, __ffs(todo) - 1);
      const uint32_t theirs = __ballot_sync(0xffffffffu, a_of == a) & 0xffffu;
      todo &= ~theirs;
      if (a != mine) fetch(a);
      const uint32_t rows16 = theirs >> (lane & 15) & 1u ? from : zeros;
      float acc[2][2][4];                            // of the two parts
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[x / 2][x % 2][e] = 0.f;
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        if (4 * k >= per) break;
        uint32_t af[2][4];
        ldmatrix4(af[1], rows16 + lo + 32 * k);
        ldmatrix4(af[0], rows16 + 32 * k);
#pragma unroll
        for (int x = 3; x >= 0; --x) mma_16816(acc[x / 2][x % 2], af[x / 2], bf[k][x % 2]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (theirs >> (g + 8 * h) & 1u) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) sum[j][2 * h + e] = acc[0][j][2 * h + e] + acc[1][j][2 * h + e];
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = __shfl_sync(0xffffffffu, row_of, g + 8 * h);
      if (p0 + g + 8 * h >= q->count[list] || base + 4 * t >= o.N) continue;
      const float back = s->back[row], f = q->factor[list][p0 + g + 8 * h];
      const uint32_t to = at(row, 16 * block + 4 * t);
      const float4 y = sm100::ld_shared_f4(to);
      sm100::st_shared_f4(to, make_float4(fmaf(f, back * sum[0][2 * h], y.x), fmaf(f, back * sum[1][2 * h], y.y),
                                          fmaf(f, back * sum[0][2 * h + 1], y.z), fmaf(f, back * sum[1][2 * h + 1], y.w)));
    }
  }
  __syncthreads();
}

}  // namespace lr
}  // namespace q4gsw
