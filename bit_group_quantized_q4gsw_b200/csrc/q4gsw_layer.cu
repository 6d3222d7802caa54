// q4gsw_layer.cu - gradients through the activations of the gated
// feed-forward block and of a projection's epilogue: the elementwise half of
// their backward passes (the products are the input-gradient kernels).
//
//   gated   d_g = d_h u act'(g),  d_u = d_h act(g)
//   linear  d_z = d_y act'(z),    d_bias[n] = sum_m d_z[m, n]
//
// Both are streams of fp16: 10 bytes per gated feature (g, u, d_h in, two
// gradients out), 6 per projected feature.  What they write the product that
// follows reads back, and at training sizes it is still in L2 then.  They are
// bound by DRAM, the small ones by filling its pipe: from cold caches 512 x 8192
// gated features (42 MB) take 10 us, 1021 x 14336 (146 MB) 26 us, 5.7 TB/s.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "q4gsw_common.cuh"
#include "q4gsw_epilogue.cuh"
#include "q4gsw_internal.h"

namespace cg = cooperative_groups;

namespace q4gsw {
namespace layer {

constexpr int kThreads = 256;
constexpr int kRows = 4;   // rows a thread of the projection's gradient has in flight

// One item a thread = 8 gated features: 32 bytes of (g, u) pairs, 16 of d_h, all
// read before any is written, so d_gu may be gu.  (As many CTAs as are resident,
// walking the items, took 0.7 us longer at 512 x 8192: the second item's loads
// waited for the first's results.)
__global__ void __launch_bounds__(kThreads) q4gsw_gated_grad_kernel(const __half* gu, const __half* d_h, __half* d_gu,
                                                                    size_t items, int act) {
  griddep_launch_dependents();
  griddep_wait();
  const size_t i = blockIdx.x * (size_t)kThreads + threadIdx.x;
  if (i >= items) return;
  const uint4 p0 = reinterpret_cast<const uint4*>(gu)[2 * i], p1 = reinterpret_cast<const uint4*>(gu)[2 * i + 1];
  const uint4 dh = reinterpret_cast<const uint4*>(d_h)[i];
  const uint32_t pw[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
  const uint32_t hw[4] = {dh.x, dh.y, dh.z, dh.w};
  uint32_t out[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 p = __half22float2(u32_as_h2(pw[j]));   // (g, u)
    const float2 d2 = __half22float2(u32_as_h2(hw[j >> 1]));
    const float d = (j & 1) ? d2.y : d2.x;
    float slope;
    const float a = act_value_slope(p.x, act, slope);
    out[j] = h2_as_u32(__floats2half2_rn(d * p.y * slope, d * a));
  }
  reinterpret_cast<uint4*>(d_gu)[2 * i] = make_uint4(out[0], out[1], out[2], out[3]);
  reinterpret_cast<uint4*>(d_gu)[2 * i + 1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// grid = (strips of 64 features, C row ranges), cluster = (1, C, 1).  Thread
// (tx, ty) walks rows ty, ty + 32, ... of its range at features 8 tx .. + 7 of
// the strip (a warp reads four 128-byte row segments); the column sums go
// over ty in shared memory, then over the C ranges through distributed shared
// memory, both in a fixed order: the same bits from every call, where atomics
// would vary.  256 x 14336 with an activation and d_bias (22 MB): 12.5 us cold;
// in ranges of 64 rows without groups of kRows rows, too few bytes were in
// flight: 16 us.  z and d_z are null without an activation;
// d_z may be z or d_y (each element is read, then written, by one thread).
__global__ void __launch_bounds__(kThreads) q4gsw_act_grad_kernel(const __half* z, const __half* d_y, __half* d_z,
                                                                  float* __restrict__ d_bias, int M, int N, int act) {
  __shared__ float part[32][65];
  __shared__ float sums[64];
  griddep_launch_dependents();
  griddep_wait();
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int C = gridDim.y, rank = blockIdx.y;
  const int n = 64 * blockIdx.x + 8 * tx;
  const int r_end = (int)((long long)(rank + 1) * M / C);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  if (n < N) {   // N % 8 == 0
    // rows in groups of kRows: all loads of a group are in flight together
    for (int r0 = (int)((long long)rank * M / C) + ty; r0 < r_end; r0 += 32 * kRows) {
      uint4 dv[kRows], zv[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int r = r0 + 32 * u;
        const size_t at = (size_t)(r < r_end ? r : r0) * N + n;
        dv[u] = *reinterpret_cast<const uint4*>(d_y + at);
        if (z) zv[u] = *reinterpret_cast<const uint4*>(z + at);
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int r = r0 + 32 * u;
        if (r >= r_end) break;
        const uint32_t dw[4] = {dv[u].x, dv[u].y, dv[u].z, dv[u].w};
        float d[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(u32_as_h2(dw[j]));
          d[2 * j] = f.x;
          d[2 * j + 1] = f.y;
        }
        if (z) {
          const uint32_t zw[4] = {zv[u].x, zv[u].y, zv[u].z, zv[u].w};
          uint32_t out[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(u32_as_h2(zw[j]));
            float s0, s1;
            act_value_slope(f.x, act, s0);
            act_value_slope(f.y, act, s1);
            d[2 * j] *= s0;
            d[2 * j + 1] *= s1;
            out[j] = h2_as_u32(__floats2half2_rn(d[2 * j], d[2 * j + 1]));
          }
          *reinterpret_cast<uint4*>(d_z + (size_t)r * N + n) = make_uint4(out[0], out[1], out[2], out[3]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += d[j];
      }
    }
  }
  if (!d_bias) return;   // the same for every thread of the launch
#pragma unroll
  for (int j = 0; j < 8; ++j) part[ty][8 * tx + j] = acc[j];
  __syncthreads();
  if (threadIdx.x < 64) {
    float s = 0.f;
    for (int y = 0; y < 32; ++y) s += part[y][threadIdx.x];
    sums[threadIdx.x] = s;
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (C > 1) cluster.sync();
  else __syncthreads();
  if (rank == 0 && threadIdx.x < 64 && 64 * blockIdx.x + threadIdx.x < N) {
    float s = sums[threadIdx.x];
    for (int q = 1; q < C; ++q) s += cluster.map_shared_rank(sums, q)[threadIdx.x];
    d_bias[64 * blockIdx.x + threadIdx.x] = s;
  }
  if (C > 1) cluster.sync();   // no CTA leaves while rank 0 reads its sums
}

}  // namespace layer

cudaError_t launch_gated_grad(const __half* gu, const __half* d_h, int M, int F, int act, __half* d_gu,
                              cudaStream_t stream) {
  const size_t items = (size_t)M * (size_t)F / 8;
  const size_t grid = (items + layer::kThreads - 1) / layer::kThreads;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(layer::kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, layer::q4gsw_gated_grad_kernel, gu, d_h, d_gu, items, act);
}

cudaError_t launch_act_grad(const __half* z, const __half* d_y, int M, int N, int act, __half* d_z, float* d_bias,
                            cudaStream_t stream) {
  const int strips = (N + 63) / 64;
  // row ranges: about two CTAs per SM, at least one group of rows in each
  const int sms = sm_count(current_device());
  int C = 1;
  while (C < 8 && (long long)strips * C < 2LL * sms && M / (2 * C) >= 32 * layer::kRows) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(strips, C, 1);
  cfg.blockDim = dim3(layer::kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = C;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, layer::q4gsw_act_grad_kernel, z, d_y, d_z, d_bias, M, N, act);
}

}  // namespace q4gsw
