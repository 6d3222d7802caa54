// q4gsw_norms.cu - the norms around a block of a decoder layer, forward and
// backward (sm_100a).
//
//   n  = block * rsqrt(mean(block^2) + eps) * (o + w_post)
//   h' = f h + gate * n
//   x  = h' * rsqrt(mean(h'^2) + eps) * (o + w_pre)
//
// A row lives in the registers of its threads from its only read to its only
// write: 8 bytes a feature forward (block, h; h', x) and 12 backward, where torch's
// elementary operations pass a row through memory for every step.  Sums, statistics
// and everything between the loads and the one rounding to fp16 are fp32.
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

struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 load8(const __half* p) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = __half22float2(u32_as_h2(w[i]));
    f.v[2 * i] = a.x;
    f.v[2 * i + 1] = a.y;
  }
  return f;
}
__device__ __forceinline__ void store8(__half* p, const F8& f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = h2_as_u32(__floats2half2_rn(f.v[2 * i], f.v[2 * i + 1]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Sums of N values over the threads of each row, the same bits in all of them.
// `buf`: [2][rows of the CTA][warps of a row][N] shared floats, used in turn.
template <int VEC, int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* buf, int& turn) {
  using R = Rows<VEC, TPR>;
#pragma unroll
  for (int o = 16; o; o /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if (R::kWarps == 1) return;
  float* b = buf + (turn * R::kPerCta + threadIdx.x / TPR) * R::kWarps * 3;
  turn ^= 1;
  const int w = threadIdx.x % TPR / 32;
  if (threadIdx.x % 32 == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[w * 3 + i] = s[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = 0.f;
#pragma unroll
    for (int k = 0; k < R::kWarps; ++k) s[i] += b[k * 3 + i];
  }
}

template <int VEC, int TPR>
__global__ void __launch_bounds__(Rows<VEC, TPR>::kThreads) q4gsw_norms_fwd_kernel(const NormsArgs a) {
  using R = Rows<VEC, TPR>;
  __shared__ float buf[2 * R::kPerCta * R::kWarps * 3];
  griddep_launch_dependents();
  griddep_wait();
  const int row = blockIdx.x * R::kPerCta + threadIdx.x / TPR;
  const int tid = threadIdx.x % TPR;
  const bool live = row < a.M;
  const size_t base = (size_t)row * a.D;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  F8 h[VEC], b[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = 8 * (tid + i * TPR);
    const bool in = live && c < a.D;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i].v[j] = b[i].v[j] = 0.f;
    if (in) h[i] = load8(a.h + base + c);
    if (in && a.block) b[i] = load8(a.block + base + c);
  }
  float r1 = 1.f;
  if (a.w_post) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(b[i].v[j], b[i].v[j], s[0]);
    row_sum<VEC, TPR, 1>(s, buf, turn);
    r1 = rsqrtf(s[0] * inv_d + a.eps);
  }
  float s2[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = 8 * (tid + i * TPR);
    if (!(live && c < a.D)) continue;
    if (a.block) {
      if (a.w_post) {
        const F8 w = load8(a.w_post + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[i].v[j] *= r1 * (a.weight_offset + w.v[j]);
      }
      if (a.gate) {
        const F8 w = load8(a.gate + (a.gate_rows ? base : 0) + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[i].v[j] *= w.v[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i].v[j] = fmaf(a.residual_scale, h[i].v[j], b[i].v[j]);
    if (a.h_out) store8(a.h_out + base + c, h[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) s2[0] = fmaf(h[i].v[j], h[i].v[j], s2[0]);
  }
  if (!a.x) return;
  row_sum<VEC, TPR, 1>(s2, buf, turn);
  const float r2 = rsqrtf(s2[0] * inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = 8 * (tid + i * TPR);
    if (!(live && c < a.D)) continue;
    const F8 w = load8(a.w_pre + c);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i].v[j] *= r2 * (a.weight_offset + w.v[j]);
    store8(a.x + base + c, h[i]);
  }
}

// Backward.  With e = d_x (o + w_pre), r2 and r1 the two norms' factors:
//   d    = d_h + r2 e - h' r2^3 mean(e h')          (the gradient of h')
//   d_h  = f d,   d_gate = d n,   p = d gate
//   d_b  = r1 p (o + w_post) - block r1^3 mean(p (o + w_post) block)
//   d_w_pre = sum of d_x h' r2,  d_w_post = sum of p block r1      over the rows
// Rows walk in steps of the grid (SUMS) and each thread adds its columns' sums in
// registers; every group of rows leaves one row of partial sums in the workspace,
// which q4gsw_norms_sum_kernel adds in a fixed order.
template <int VEC, int TPR, bool SUMS>
__global__ void __launch_bounds__(Rows<VEC, TPR>::kThreads) q4gsw_norms_bwd_kernel(const NormsArgs a) {
  using R = Rows<VEC, TPR>;
  __shared__ float buf[2 * R::kPerCta * R::kWarps * 3];
  griddep_launch_dependents();
  griddep_wait();
  const int group = blockIdx.x * R::kPerCta + threadIdx.x / TPR, groups = gridDim.x * R::kPerCta;
  const int tid = threadIdx.x % TPR;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  F8 wpre[SUMS ? VEC : 1], wpost[SUMS ? VEC : 1], wgate[SUMS ? VEC : 1];
  if (SUMS) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) wpre[i].v[j] = wpost[i].v[j] = wgate[i].v[j] = 0.f;
  }
  // every group of a CTA takes the same number of turns: they share its barriers
  const int turns = (a.M + groups - 1) / groups;
  for (int u = 0; u < turns; ++u) {
    const int row = group + u * groups;
    const bool live = row < a.M;
    const size_t base = (size_t)row * a.D;
    F8 h[VEC], d[VEC], b[VEC], dx[VEC];
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = 8 * (tid + i * TPR);
      const bool in = live && c < a.D;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i].v[j] = d[i].v[j] = b[i].v[j] = dx[i].v[j] = 0.f;
      if (!in) continue;
      if (a.d_x) {
        h[i] = load8(a.h + base + c);
        dx[i] = load8(a.d_x + base + c);
      }
      if (a.d_h) d[i] = load8(a.d_h + base + c);
      if (a.block) b[i] = load8(a.block + base + c);
      if (a.d_x) {
        const F8 w = load8(a.w_pre + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[0] = fmaf(h[i].v[j], h[i].v[j], s[0]);
          s[1] = fmaf(dx[i].v[j] * (a.weight_offset + w.v[j]), h[i].v[j], s[1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[2] = fmaf(b[i].v[j], b[i].v[j], s[2]);
    }
    row_sum<VEC, TPR, 3>(s, buf, turn);
    const float r2 = rsqrtf(s[0] * inv_d + a.eps), r1 = a.w_post ? rsqrtf(s[2] * inv_d + a.eps) : 1.f;
    const float pull = r2 * r2 * r2 * (s[1] * inv_d);
    float s4[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = 8 * (tid + i * TPR);
      if (!(live && c < a.D)) continue;
      if (a.d_x) {
        const F8 w = load8(a.w_pre + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          d[i].v[j] += r2 * (dx[i].v[j] * (a.weight_offset + w.v[j])) - pull * h[i].v[j];
          if (SUMS) wpre[i].v[j] = fmaf(dx[i].v[j] * h[i].v[j], r2, wpre[i].v[j]);
        }
      }
      F8 out;
#pragma unroll
      for (int j = 0; j < 8; ++j) out.v[j] = a.residual_scale * d[i].v[j];
      store8(a.h_out + base + c, out);
      if (!a.block) continue;
      F8 w;
#pragma unroll
      for (int j = 0; j < 8; ++j) w.v[j] = 1.f;
      if (a.w_post) {
        w = load8(a.w_post + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) w.v[j] += a.weight_offset;
      }
      if (a.gate) {
        const F8 gate = load8(a.gate + (a.gate_rows ? base : 0) + c);
        F8 dg;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dg.v[j] = d[i].v[j] * (b[i].v[j] * (r1 * w.v[j]));
          if (SUMS) wgate[i].v[j] += dg.v[j];
          d[i].v[j] *= gate.v[j];
        }
        if (a.gate_rows) store8(a.d_gate_rows + base + c, dg);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (SUMS) wpost[i].v[j] = fmaf(d[i].v[j] * b[i].v[j], r1, wpost[i].v[j]);
        d[i].v[j] *= w.v[j];
        s4[0] = fmaf(d[i].v[j], b[i].v[j], s4[0]);
      }
    }
    if (!a.block) continue;
    float pull_b = 0.f;
    if (a.w_post) {
      row_sum<VEC, TPR, 1>(s4, buf, turn);
      pull_b = r1 * r1 * r1 * (s4[0] * inv_d);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = 8 * (tid + i * TPR);
      if (!(live && c < a.D)) continue;
      F8 out;
#pragma unroll
      for (int j = 0; j < 8; ++j) out.v[j] = r1 * d[i].v[j] - pull_b * b[i].v[j];
      store8(a.x + base + c, out);
    }
  }
  if (!SUMS) return;
#pragma unroll
  for (int i = 0; i < (SUMS ? VEC : 1); ++i) {
    const int c = 8 * (tid + i * TPR);
    if (c >= a.D) continue;
    float* p = a.part + (size_t)group * 3 * a.D + c;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = wpre[i].v[j];
      p[a.D + j] = wpost[i].v[j];
      p[2 * a.D + j] = wgate[i].v[j];
    }
  }
}

constexpr int kSumColumns = 32, kSumRows = 8;

// grid (columns / 32, 3): one of the three sums over the groups' partial rows
__global__ void __launch_bounds__(kSumColumns * kSumRows)
q4gsw_norms_sum_kernel(const float* part, int groups, int D, float* d_w_pre, float* d_w_post, float* d_gate) {
  __shared__ float s_part[kSumRows][kSumColumns];
  griddep_launch_dependents();
  griddep_wait();
  float* out = blockIdx.y == 0 ? d_w_pre : blockIdx.y == 1 ? d_w_post : d_gate;
  if (!out) return;
  const int x = threadIdx.x % kSumColumns, y = threadIdx.x / kSumColumns;
  const int c = blockIdx.x * kSumColumns + x;
  float s = 0.f;
  if (c < D)
    for (int p = y; p < groups; p += kSumRows) s += part[((size_t)p * 3 + blockIdx.y) * D + c];
  s_part[y][x] = s;
  __syncthreads();
  if (y == 0 && c < D) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kSumRows; ++k) s += s_part[k][x];
    out[c] = s;
  }
}

// CTAs that leave partial sums: two per SM of the largest part (a constant, so that
// the workspace's size is a function of M and D)
constexpr int kSumGroups = 296;

struct Shape {
  int vec, tpr;
};
// 8 features a thread up to 1024 threads, then two and four vectors of 8
inline Shape shape_of(int D) {
  const int nv = (D + 7) / 8;
  if (nv <= 32) return {1, 32};
  if (nv <= 128) return {1, 128};
  if (nv <= 256) return {1, 256};
  if (nv <= 512) return {1, 512};
  if (nv <= 1024) return {1, 1024};
  if (nv <= 2048) return {2, 1024};
  return {4, 1024};
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

template <int VEC, int TPR>
static cudaError_t norms_bwd_rows(const NormsArgs& a, cudaStream_t stream) {
  using R = norms::Rows<VEC, TPR>;
  cudaLaunchAttribute attr[1];
  int ctas = (a.M + R::kPerCta - 1) / R::kPerCta;
  if (!a.part) {
    const cudaLaunchConfig_t cfg = norms_config(attr, ctas, R::kThreads, stream);
    return cudaLaunchKernelEx(&cfg, norms::q4gsw_norms_bwd_kernel<VEC, TPR, false>, a);
  }
  ctas = ctas < norms::kSumGroups / R::kPerCta ? ctas : norms::kSumGroups / R::kPerCta;
  cudaLaunchConfig_t cfg = norms_config(attr, ctas, R::kThreads, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norms::q4gsw_norms_bwd_kernel<VEC, TPR, true>, a);
  if (e != cudaSuccess) return e;
  cfg = norms_config(attr, (a.D + norms::kSumColumns - 1) / norms::kSumColumns, norms::kSumColumns * norms::kSumRows,
                     stream);
  cfg.gridDim.y = 3;
  return cudaLaunchKernelEx(&cfg, norms::q4gsw_norms_sum_kernel, (const float*)a.part, ctas * R::kPerCta, a.D,
                            a.d_w_pre, a.d_w_post, a.d_gate);
}

#define Q4_NORMS(FN)                                                              \
  do {                                                                            \
    if (s.vec == 4) return FN<4, 1024>(a, stream);                                \
    if (s.vec == 2) return FN<2, 1024>(a, stream);                                \
    switch (s.tpr) {                                                              \
      case 32: return FN<1, 32>(a, stream);                                       \
      case 128: return FN<1, 128>(a, stream);                                     \
      case 256: return FN<1, 256>(a, stream);                                     \
      case 512: return FN<1, 512>(a, stream);                                     \
      default: return FN<1, 1024>(a, stream);                                     \
    }                                                                             \
  } while (0)

size_t norms_workspace_bytes(int M, int D) {
  // a group of rows each: at most kSumGroups, and no more than there are rows rounded
  // up to a CTA's four
  const long long groups = (M + 3LL) / 4 * 4;
  return sizeof(float) * 3 * (size_t)D * (size_t)(groups < norms::kSumGroups ? groups : norms::kSumGroups);
}

cudaError_t launch_norms_fwd(const NormsArgs& a, cudaStream_t stream, char* route, int route_len) {
  const norms::Shape s = norms::shape_of(a.D);
  snprintf(route, route_len, "norms_fwd launches=1 threads=%d vec=%d", s.tpr, s.vec);
  Q4_NORMS(norms_fwd_rows);
}

cudaError_t launch_norms_bwd(const NormsArgs& a, cudaStream_t stream, char* route, int route_len) {
  const norms::Shape s = norms::shape_of(a.D);
  snprintf(route, route_len, "norms_bwd launches=%d threads=%d vec=%d", a.part ? 2 : 1, s.tpr, s.vec);
  Q4_NORMS(norms_bwd_rows);
}

}  // namespace q4gsw
