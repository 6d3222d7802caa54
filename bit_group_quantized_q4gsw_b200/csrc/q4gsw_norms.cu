// q4gsw_norms.cu - the norms around a block of a decoder layer, forward and
// backward (sm_100a).
//
//   n  = block * rsqrt(mean(block^2) + eps) * (o + w_post)
//   h' = f h + gate * n
//   x  = h' * rsqrt(mean(h'^2) + eps) * (o + w_pre)
//
// A row lives in the registers of its threads from its only read to its only
// write: 8 bytes a feature forward (block, h; h', x) and 12 backward, where elementary
// operations pass a row through memory for every step.  Sums, statistics and everything
// between the loads and the one rounding to fp16 are fp32.  Forward, 4096 x 4096: 24.5
// us, 84 % of the copy rate; 1 x 2048: 2.1 us, a launch and two dependent rounds of loads.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdio>

#include "q4gsw_common.cuh"
#include "q4gsw_internal.h"

namespace q4gsw {
namespace norms {

// TPR threads to a row, VEC vectors of 8 features each; rows of up to 128 threads
// share a CTA of 128.
template <int VEC, int TPR>
struct Rows {
  static constexpr int kThreads = TPR < 128 ? 128 : TPR;
  static constexpr int kPerCta = kThreads / TPR;
  static constexpr int kWarps = TPR / 32;        // warps of a row
};

// 8 features as they lie in memory (4 registers), widened where they are used
__device__ __forceinline__ uint4 load8(const __half* p) { return *reinterpret_cast<const uint4*>(p); }
// Eight features as four pairs: the packed fp32 instructions work on two values at
// once, and these kernels are bound by the instructions they issue.
struct V8 {
  unsigned long long p[4];
};
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long both(float v) { return pack2(v, v); }
__device__ __forceinline__ V8 widen(const uint4& r) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  V8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(u32_as_h2(w[i]));
    v.p[i] = pack2(f.x, f.y);
  }
  return v;
}
__device__ __forceinline__ void store8(__half* p, const V8& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(v.p[i]);
    w[i] = h2_as_u32(__floats2half2_rn(f.x, f.y));
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// offset + w of 8 features
__device__ __forceinline__ V8 weights8(const __half* p, float offset) {
  V8 v = widen(load8(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(v.p[i]);
    v.p[i] = pack2(offset + f.x, offset + f.y);
  }
  return v;
}
__device__ __forceinline__ V8 ones8() { return V8{{both(1.f), both(1.f), both(1.f), both(1.f)}}; }
__device__ __forceinline__ float add_up(unsigned long long v) {
  const float2 f = unpack2(v);
  return f.x + f.y;
}

// Sums over the threads of each row, the same bits in all of them: over the lanes of
// a warp, through `buf` ([2][rows of the CTA][N][warps of a row] shared floats, used in
// turn) over the warps, whose sums the lanes of every warp add between them.  Three
// sums share the steps: after two halvings each group of eight lanes has one of them
// (6 shuffles where three butterflies take 15).
template <class R>
__host__ __device__ constexpr int row_sum_floats() {
  return 2 * R::kPerCta * 3 * R::kWarps;
}
template <int FROM>
__device__ __forceinline__ float butterfly(float v) {
#pragma unroll
  for (int o = FROM; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <class R>
__device__ __forceinline__ float row_sum(float s, float* buf, int& turn) {
  s = butterfly<16>(s);
  if (R::kWarps == 1) return s;
  constexpr int TPR = 32 * R::kWarps;
  float* b = buf + (turn * R::kPerCta + threadIdx.x / TPR) * 3 * R::kWarps;
  turn ^= 1;
  if (threadIdx.x % 32 == 0) b[threadIdx.x % TPR / 32] = s;
  __syncthreads();
  return butterfly<R::kWarps / 2>(b[threadIdx.x % R::kWarps]);
}
template <class R>
__device__ __forceinline__ void row_sum3(float (&s)[3], float* buf, int& turn) {
  const int lane = threadIdx.x % 32;
  const bool up = lane & 16, odd = lane & 8;
  // lanes 0-15: s0 and s1, lanes 16-31: s2
  float v = (up ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, up ? s[0] : s[2], 16);
  const float w = (up ? 0.f : s[1]) + __shfl_xor_sync(0xffffffffu, up ? s[1] : 0.f, 16);
  v = (odd ? w : v) + __shfl_xor_sync(0xffffffffu, odd ? v : w, 8);
  v = butterfly<4>(v);                  // lanes 0-7: s0, 8-15: s1, 16-23: s2
  if constexpr (R::kWarps > 1) {
    constexpr int TPR = 32 * R::kWarps, W = R::kWarps;
    float* b = buf + (turn * R::kPerCta + threadIdx.x / TPR) * 3 * W;
    turn ^= 1;
    if (lane % 8 == 0 && lane < 24) b[lane / 8 * W + threadIdx.x % TPR / 32] = v;
    __syncthreads();
    const float* mine = b + min(lane / 8, 2) * W;
    constexpr int S = W < 8 ? W : 8;
    v = mine[lane % S];
#pragma unroll
    for (int k = 8; k < W; k += 8) v += mine[lane % 8 + k];
    v = butterfly<S / 2>(v);
  }
  s[0] = __shfl_sync(0xffffffffu, v, 0);
  s[1] = __shfl_sync(0xffffffffu, v, 8);
  s[2] = __shfl_sync(0xffffffffu, v, 16);
}

template <int VEC, int TPR>
__global__ void __launch_bounds__(Rows<VEC, TPR>::kThreads) q4gsw_norms_fwd_kernel(const NormsArgs a) {
  using R = Rows<VEC, TPR>;
  __shared__ float buf[row_sum_floats<R>()];
  griddep_launch_dependents();
  griddep_wait();
  const int row = blockIdx.x * R::kPerCta + threadIdx.x / TPR;
  const int tid = threadIdx.x % TPR;
  const bool live = row < a.M;
  const size_t base = (size_t)row * a.D;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  uint4 h[VEC], b[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = 8 * (tid + i * TPR);
    const bool in = live && c < a.D;
    h[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (in) h[i] = load8(a.h + base + c);
    if (in && a.block) b[i] = load8(a.block + base + c);
  }
  float r1 = 1.f;
  if (a.w_post) {
    unsigned long long q = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const V8 f = widen(b[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) q = fma2(f.p[j], f.p[j], q);
    }
    r1 = rsqrtf(row_sum<R>(add_up(q), buf, turn) * inv_d + a.eps);
  }
  V8 v[VEC];      // h'
  unsigned long long q = 0;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = 8 * (tid + i * TPR);
    if (!(live && c < a.D)) continue;
    V8 n = widen(b[i]);
    if (a.w_post) {
      const V8 w = weights8(a.w_post + c, a.weight_offset);
#pragma unroll
      for (int j = 0; j < 4; ++j) n.p[j] = mul2(n.p[j], mul2(both(r1), w.p[j]));
    }
    if (a.gate) {
      const V8 w = widen(load8(a.gate + (a.gate_rows ? base : 0) + c));
#pragma unroll
      for (int j = 0; j < 4; ++j) n.p[j] = mul2(n.p[j], w.p[j]);
    }
    v[i] = widen(h[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[i].p[j] = fma2(both(a.residual_scale), v[i].p[j], n.p[j]);
      q = fma2(v[i].p[j], v[i].p[j], q);
    }
    if (a.h_out) store8(a.h_out + base + c, v[i]);
  }
  if (!a.x) return;
  const float r2 = rsqrtf(row_sum<R>(add_up(q), buf, turn) * inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = 8 * (tid + i * TPR);
    if (!(live && c < a.D)) continue;
    const V8 w = weights8(a.w_pre + c, a.weight_offset);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i].p[j] = mul2(v[i].p[j], mul2(both(r2), w.p[j]));
    store8(a.x + base + c, v[i]);
  }
}

// Backward.  With e = d_x (o + w_pre), r2 and r1 the two norms' factors:
//   d    = d_h + r2 e - h' r2^3 mean(e h')          (the gradient of h')
//   d_h  = f d,   d_gate = d n,   p = d gate
//   d_b  = r1 p (o + w_post) - block r1^3 mean(p (o + w_post) block)
//   d_w_pre = sum of d_x h' r2,  d_w_post = sum of p block r1      over the rows
// As many CTAs as are resident walk the rows in steps of the grid.  With STAGES > 0
// each thread copies its own vectors of the row that is STAGES turns ahead into its own
// slots of shared memory (cp.async; no thread reads another's, so no barrier is needed),
// and memory is busy while a row is reduced.  SUMS: each thread adds its columns' sums
// over its rows in registers, every CTA leaves one row of partial sums in the
// workspace, and q4gsw_norms_sum_kernel adds those in a fixed order.
//
// Bound by issued instructions as much as by bytes: 4096 x 4096 took 93 us with scalar
// arithmetic on eight widened features a thread, 61 with the ring, 48 with packed pairs
// and the columns' weights kept in registers, 44 with the shared butterfly of row_sum3
// (30.7 us at the copy rate).  1021 x 4096: 13.9; 512 x 2048 with the three sums: 10.5,
// two launches of which the sums are 3.
template <int VEC, int TPR, bool SUMS>
struct BwdRows {
  // with sums, CTAs of 512 threads or more: fewer partial rows for the launch behind
  static constexpr int kThreads = SUMS ? (TPR < 512 ? 512 : TPR) : Rows<VEC, TPR>::kThreads;
  static constexpr int kPerCta = kThreads / TPR;
  static constexpr int kWarps = TPR / 32;
  static constexpr int kMinCtas = SUMS || kThreads == 1024 ? 1 : 1024 / kThreads / (VEC > 1 ? 2 : 1);
};

template <int VEC, int TPR, bool SUMS, int STAGES>
__global__ void __launch_bounds__(BwdRows<VEC, TPR, SUMS>::kThreads, BwdRows<VEC, TPR, SUMS>::kMinCtas)
q4gsw_norms_bwd_kernel(const NormsArgs a) {
  using R = BwdRows<VEC, TPR, SUMS>;
  __shared__ float buf[row_sum_floats<R>()];
  extern __shared__ uint4 ring[];      // [STAGES][operands in use][VEC][kThreads]
  griddep_launch_dependents();
  griddep_wait();
  const int sub = threadIdx.x / TPR;
  const int group = blockIdx.x * R::kPerCta + sub, groups = gridDim.x * R::kPerCta;
  const int tid = threadIdx.x % TPR;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  V8 sum[SUMS ? 3 : 1][SUMS ? VEC : 1];      // d_w_pre, d_w_post, d_gate of this thread's columns
  if (SUMS) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[k][i] = V8{{0, 0, 0, 0}};
  }
  // the weights of this thread's columns, 1 where there are none, are the same for
  // every row: one vector a thread keeps them in registers, more read them again
  constexpr bool kKeep = VEC == 1;
  V8 w_pre[kKeep ? 1 : VEC], w_post[kKeep ? 1 : VEC], w_gate[kKeep ? 1 : VEC];
  auto weight = [&](const __half* p, int i, float offset) {
    const int c = 8 * (tid + i * TPR);
    return c < a.D && p ? weights8(p + c, offset) : ones8();
  };
  const __half* feature_gate = a.gate && !a.gate_rows ? a.gate : nullptr;
  if constexpr (kKeep) {
    w_pre[0] = weight(a.w_pre, 0, a.weight_offset);
    w_post[0] = weight(a.w_post, 0, a.weight_offset);
    w_gate[0] = weight(feature_gate, 0, 0.f);
  }
  // every group of a CTA takes the same number of turns: they share its barriers
  const int turns = (int)(((long long)a.M + groups - 1) / groups);
  const bool gate_rows = a.gate && a.gate_rows;
  const int ring_h = 0, ring_dx = VEC, ring_dh = a.d_x ? 2 * VEC : 0, ring_b = ring_dh + (a.d_h ? VEC : 0),
            ring_g = ring_b + (a.block ? VEC : 0), ring_all = ring_g + (gate_rows ? VEC : 0);
  auto fetch = [&](int u) {     // this thread's vectors of turn u into its slot
    const int row = group + u * groups;
    if (u < turns && row < a.M) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int c = 8 * (tid + i * TPR);
        if (c >= a.D) continue;
        const size_t at = (size_t)row * a.D + c;
        const uint32_t slot = (uint32_t)__cvta_generic_to_shared(ring) +
                              16u * (uint32_t)(((u % (STAGES ? STAGES : 1)) * ring_all + i) * R::kThreads + (int)threadIdx.x);
        const uint32_t step = 16u * R::kThreads;
        if (a.d_x) {
          cp_async_16(slot + step * ring_h, a.h + at);
          cp_async_16(slot + step * ring_dx, a.d_x + at);
        }
        if (a.d_h) cp_async_16(slot + step * ring_dh, a.d_h + at);
        if (a.block) cp_async_16(slot + step * ring_b, a.block + at);
        if (gate_rows) cp_async_16(slot + step * ring_g, a.gate + at);
      }
    }
    cp_async_commit();
  };
  if constexpr (STAGES > 0) {
    for (int u = 0; u < STAGES; ++u) fetch(u);
  }
  for (int u = 0; u < turns; ++u) {
    const int row = group + u * groups;
    const bool live = row < a.M;
    const size_t base = (size_t)row * a.D;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4* slot = ring + (size_t)(u % (STAGES ? STAGES : 1)) * ring_all * R::kThreads + threadIdx.x;
    if constexpr (STAGES > 0) cp_async_wait<STAGES - 1>();
    uint4 h[VEC], dh[VEC], b[VEC], dx[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = 8 * (tid + i * TPR);
      const bool in = live && c < a.D;
      auto get = [&](const __half* p, int at) { return STAGES ? slot[(at + i) * R::kThreads] : load8(p + base + c); };
      h[i] = in && a.d_x ? get(a.h, ring_h) : zero;
      dx[i] = in && a.d_x ? get(a.d_x, ring_dx) : zero;
      dh[i] = in && a.d_h ? get(a.d_h, ring_dh) : zero;
      b[i] = in && a.block ? get(a.block, ring_b) : zero;
    }
    V8 hv[VEC], bv[VEC], d[VEC];
    unsigned long long q0 = 0, q1 = 0, q2 = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      hv[i] = widen(h[i]);
      bv[i] = widen(b[i]);
      d[i] = widen(dx[i]);
      if (!kKeep) w_pre[i] = weight(a.w_pre, i, a.weight_offset);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned long long e = mul2(d[i].p[j], w_pre[i].p[j]);
        q0 = fma2(hv[i].p[j], hv[i].p[j], q0);
        q1 = fma2(e, hv[i].p[j], q1);
        q2 = fma2(bv[i].p[j], bv[i].p[j], q2);
      }
    }
    float s[3] = {add_up(q0), add_up(q1), add_up(q2)};
    row_sum3<R>(s, buf, turn);
    const float r2 = rsqrtf(s[0] * inv_d + a.eps), r1 = a.w_post ? rsqrtf(s[2] * inv_d + a.eps) : 1.f;
    // (in this order: a row of zeros has no pull, however large its factor's cube is)
    const float pull = a.d_x ? r2 * (r2 * (r2 * (s[1] * inv_d))) : 0.f;
    unsigned long long q4 = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = 8 * (tid + i * TPR);
      if (!(live && c < a.D)) continue;
      const V8 dhv = widen(dh[i]);
      if (!kKeep) {
        w_pre[i] = weight(a.w_pre, i, a.weight_offset);
        w_post[i] = weight(a.w_post, i, a.weight_offset);
        w_gate[i] = weight(feature_gate, i, 0.f);
      }
      V8 out;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned long long k = mul2(d[i].p[j], both(a.d_x ? r2 : 0.f));
        if (SUMS) sum[0][i].p[j] = fma2(k, hv[i].p[j], sum[0][i].p[j]);
        d[i].p[j] = fma2(both(-pull), hv[i].p[j], fma2(k, w_pre[i].p[j], dhv.p[j]));
        out.p[j] = mul2(both(a.residual_scale), d[i].p[j]);
      }
      store8(a.h_out + base + c, out);
      if (!a.block) continue;
      if (a.gate) {
        const V8 gate = !gate_rows ? w_gate[i]
                                   : widen(STAGES ? slot[(ring_g + i) * R::kThreads] : load8(a.gate + base + c));
        V8 dg;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dg.p[j] = mul2(d[i].p[j], mul2(bv[i].p[j], mul2(both(r1), w_post[i].p[j])));
          if (SUMS) sum[2][i].p[j] = fma2(both(1.f), dg.p[j], sum[2][i].p[j]);
          d[i].p[j] = mul2(d[i].p[j], gate.p[j]);
        }
        if (gate_rows) store8(a.d_gate_rows + base + c, dg);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (SUMS) sum[1][i].p[j] = fma2(mul2(d[i].p[j], both(r1)), bv[i].p[j], sum[1][i].p[j]);
        d[i].p[j] = mul2(d[i].p[j], w_post[i].p[j]);
        q4 = fma2(d[i].p[j], bv[i].p[j], q4);
      }
    }
    if constexpr (STAGES > 0) fetch(u + STAGES);      // every vector of the slot is in registers or used
    if (!a.block) continue;
    float pull_b = 0.f;
    if (a.w_post) {
      pull_b = r1 * (r1 * (r1 * (row_sum<R>(add_up(q4), buf, turn) * inv_d)));
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = 8 * (tid + i * TPR);
      if (!(live && c < a.D)) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) d[i].p[j] = fma2(both(-pull_b), bv[i].p[j], mul2(both(r1), d[i].p[j]));
      store8(a.x + base + c, d[i]);
    }
  }
  if (!SUMS) return;
  // the CTA's groups of rows, then one row of partial sums
  if constexpr (SUMS) {
    if constexpr (R::kPerCta > 1) {
      __shared__ V8 other[R::kPerCta - 1][TPR];
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          __syncthreads();
          if (sub) other[sub - 1][tid] = sum[k][i];
          __syncthreads();
          if (!sub)
#pragma unroll
            for (int q = 0; q < R::kPerCta - 1; ++q) {
              const V8 x = other[q][tid];
#pragma unroll
              for (int j = 0; j < 4; ++j) sum[k][i].p[j] = fma2(both(1.f), x.p[j], sum[k][i].p[j]);
            }
        }
      if (sub) return;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = 8 * (tid + i * TPR);
      if (c >= a.D) continue;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        ulonglong2* p = reinterpret_cast<ulonglong2*>(a.part + ((size_t)blockIdx.x * 3 + k) * a.D + c);
        p[0] = make_ulonglong2(sum[k][i].p[0], sum[k][i].p[1]);
        p[1] = make_ulonglong2(sum[k][i].p[2], sum[k][i].p[3]);
      }
    }
  }
}

constexpr int kSumColumns = 32, kSumRows = 32;

// grid (columns / 32, 3): one of the three sums over the CTAs' partial rows
__global__ void __launch_bounds__(kSumColumns * kSumRows)
q4gsw_norms_sum_kernel(const float* part, int parts, int D, float* d_w_pre, float* d_w_post, float* d_gate) {
  __shared__ float s_part[kSumRows][kSumColumns + 1];
  griddep_launch_dependents();
  griddep_wait();
  float* out = blockIdx.y == 0 ? d_w_pre : blockIdx.y == 1 ? d_w_post : d_gate;
  if (!out) return;
  const int x = threadIdx.x % kSumColumns, y = threadIdx.x / kSumColumns;
  const int c = blockIdx.x * kSumColumns + x;
  float s = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int p = y; p < parts; p += kSumRows) s += part[((size_t)p * 3 + blockIdx.y) * D + c];
  }
  s_part[y][x] = s;
  __syncthreads();
  // warp y adds the rows of column y
  s = s_part[x][y];
#pragma unroll
  for (int o = 16; o; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (x == 0 && blockIdx.x * kSumColumns + y < D) out[blockIdx.x * kSumColumns + y] = s;
}

// CTAs that leave partial sums, at most (a constant, so that the workspace's size
// is a function of M and D)
constexpr int kSumCtas = 148;
// shared memory of a ring: what a CTA may have beside the static part
constexpr int kMaxRing = 208 * 1024;

// Threads to a row and vectors of 8 features to a thread.  One vector where there are
// few rows (the row's latency counts: 1 x 2048 forward 2.1 us, 2.5 with two) and in the
// backward pass, whose registers hold the columns' weights then (4096 x 4096: 44.1 us,
// 50.4 with two); two in the forward from 2^21 features on (4096 x 4096: 24.5 us, 28.4
// with one); four beyond 8192 features (1000 x 16384: forward 27.3 us, 36.8 with two;
// backward 60.9 and 65.7).  Beyond 8192 features the backward pass keeps four vectors of
// three rows and their weights and spills: 152 to 172 bytes a thread of stores with 512
// threads, 624 to 712 with 1024, and 1296 to 2692 with the sums, whose columns it holds
// too; with the sums 1024 threads of one vector spill 208 to 220.  1000 rows, backward
// and with all three sums (us; the floor of both in brackets): 4096 features 13.0 and
// 19.0 (7.5), 8192 24.1 and 47.5 (15), 12288 49.6 and 88.0 (22.5), 16384 60.9 and 124
// (30), 32768 213 and 390 (60).
struct Shape {
  int vec, tpr;
};
inline Shape shape_of(int D, int M, bool fwd) {
  const int nv = D / 8;
  int vec = nv > 1024 ? 4 : fwd && nv > 32 && (long long)M * D >= (1 << 21) ? 2 : 1;
  int tpr = vec == 4 ? 512 : 32;
  while (tpr * vec < nv) tpr *= 2;
  return {vec, tpr};
}

}  // namespace norms

static cudaLaunchConfig_t norms_config(cudaLaunchAttribute* attr, int grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int VEC, int TPR>
static cudaError_t norms_fwd_rows(const NormsArgs& a, cudaStream_t stream) {
  using R = norms::Rows<VEC, TPR>;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = norms_config(attr, (a.M + R::kPerCta - 1) / R::kPerCta, R::kThreads, stream);
  return cudaLaunchKernelEx(&cfg, norms::q4gsw_norms_fwd_kernel<VEC, TPR>, a);
}

template <int VEC, int TPR, bool SUMS, int STAGES>
static cudaError_t norms_bwd_launch(const NormsArgs& a, int ctas, size_t ring, cudaStream_t stream) {
  auto kernel = norms::q4gsw_norms_bwd_kernel<VEC, TPR, SUMS, STAGES>;
  static PerDeviceOnce once;
  const cudaError_t e = once_per_device(once, current_device(), [&] {
    return STAGES ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, norms::kMaxRing) : cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = norms_config(attr, ctas, norms::BwdRows<VEC, TPR, SUMS>::kThreads, stream);
  cfg.dynamicSmemBytes = ring * STAGES;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int VEC, int TPR, bool SUMS>
static cudaError_t norms_bwd_form(const NormsArgs& a, cudaStream_t stream, int* parts) {
  using R = norms::BwdRows<VEC, TPR, SUMS>;
  const int operands = (a.d_x ? 2 : 0) + (a.d_h ? 1 : 0) + (a.block ? 1 : 0) + (a.gate && a.gate_rows ? 1 : 0);
  const size_t ring = sizeof(uint4) * (size_t)operands * VEC * R::kThreads;
  const long long rows = ((long long)a.M + R::kPerCta - 1) / R::kPerCta;
  int per_sm = R::kMinCtas;
  while (per_sm > 1 && per_sm * 2 * ring > norms::kMaxRing) --per_sm;
  const long long most = SUMS ? norms::kSumCtas : (long long)per_sm * sm_count(current_device());
  const int ctas = (int)(rows < most ? rows : most);
  *parts = ctas;
  // Rows beyond what is resident at once are fetched a turn ahead (4096 x 4096: 44.1 us,
  // 53.0 without); where two slots do not fit, every row has a CTA of its own.
  if (rows <= ctas || 2 * ring > norms::kMaxRing)
    return norms_bwd_launch<VEC, TPR, SUMS, 0>(a, SUMS ? ctas : (int)rows, 0, stream);
  return norms_bwd_launch<VEC, TPR, SUMS, 2>(a, ctas, ring, stream);
}

template <int VEC, int TPR>
static cudaError_t norms_bwd_rows(const NormsArgs& a, cudaStream_t stream) {
  int parts = 0;
  if (!a.part) return norms_bwd_form<VEC, TPR, false>(a, stream, &parts);
  const cudaError_t e = norms_bwd_form<VEC, TPR, true>(a, stream, &parts);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = norms_config(attr, (a.D + norms::kSumColumns - 1) / norms::kSumColumns,
                                        norms::kSumColumns * norms::kSumRows, stream);
  cfg.gridDim.y = 3;
  return cudaLaunchKernelEx(&cfg, norms::q4gsw_norms_sum_kernel, (const float*)a.part, parts, a.D, a.d_w_pre,
                            a.d_w_post, a.d_gate);
}

size_t norms_workspace_bytes(int M, int D) {
  return sizeof(float) * 3 * (size_t)D * (size_t)(M < norms::kSumCtas ? M : norms::kSumCtas);
}

cudaError_t launch_norms_fwd(const NormsArgs& a, cudaStream_t stream, char* route, int route_len) {
  const norms::Shape s = norms::shape_of(a.D, a.M, true);
  snprintf(route, route_len, "norms_fwd launches=1 threads=%d vec=%d", s.tpr, s.vec);
  if (s.vec == 4) return s.tpr == 512 ? norms_fwd_rows<4, 512>(a, stream) : norms_fwd_rows<4, 1024>(a, stream);
  if (s.vec == 2) {
    switch (s.tpr) {
      case 32: return norms_fwd_rows<2, 32>(a, stream);
      case 64: return norms_fwd_rows<2, 64>(a, stream);
      case 128: return norms_fwd_rows<2, 128>(a, stream);
      case 256: return norms_fwd_rows<2, 256>(a, stream);
      default: return norms_fwd_rows<2, 512>(a, stream);
    }
  }
  switch (s.tpr) {
    case 32: return norms_fwd_rows<1, 32>(a, stream);
    case 64: return norms_fwd_rows<1, 64>(a, stream);
    case 128: return norms_fwd_rows<1, 128>(a, stream);
    case 256: return norms_fwd_rows<1, 256>(a, stream);
    case 512: return norms_fwd_rows<1, 512>(a, stream);
    default: return norms_fwd_rows<1, 1024>(a, stream);
  }
}

cudaError_t launch_norms_bwd(const NormsArgs& a, cudaStream_t stream, char* route, int route_len) {
  const norms::Shape s = norms::shape_of(a.D, a.M, false);
  snprintf(route, route_len, "norms_bwd launches=%d threads=%d vec=%d", a.part ? 2 : 1, s.tpr, s.vec);
  if (s.vec == 4) return s.tpr == 512 ? norms_bwd_rows<4, 512>(a, stream) : norms_bwd_rows<4, 1024>(a, stream);
  switch (s.tpr) {
    case 32: return norms_bwd_rows<1, 32>(a, stream);
    case 64: return norms_bwd_rows<1, 64>(a, stream);
    case 128: return norms_bwd_rows<1, 128>(a, stream);
    case 256: return norms_bwd_rows<1, 256>(a, stream);
    case 512: return norms_bwd_rows<1, 512>(a, stream);
    default: return norms_bwd_rows<1, 1024>(a, stream);
  }
}

}  // namespace q4gsw
