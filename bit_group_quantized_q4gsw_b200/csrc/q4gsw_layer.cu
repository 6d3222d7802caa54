// q4gsw_layer.cu - gradients through the activations of the gated
// feed-forward block and of a projection's epilogue: the elementwise half of
// their backward passes (the products are the input-gradient kernels).
//
//   gated   d_g = d_h u act'(g),  d_u = d_h act(g)
//   linear  d_z = d_y act'(z),    d_bias[n] = sum_m d_z[m, n]
//
// Both are streams of fp16: 10 bytes per gated feature (g, u, d_h in, two
// gradients out), 6 per projected feature.  What they write the product that
// follows reads back, and at training sizes it is still in L2 then.  From cold
// caches 1021 x 14336 gated features (146 MB) take 19.8 us, bound by DRAM (66 % of
// its rate, writes in L2 apart); 512 x 8192 (42 MB) 9.3 us and 256 x 14336 projected
// features (22 MB) 10.6 us at 33 and 17 %, bound by the latency of one or two
// dependent rounds of loads.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "q4gsw_common.cuh"
#include "q4gsw_epilogue.cuh"
#include "q4gsw_internal.h"

namespace cg = cooperative_groups;

namespace q4gsw {
namespace layer {

constexpr int kThreads = 256;
constexpr int kItems = 2;   // items a thread of the gated gradient has in flight

// One item = 4 gated features: 16 bytes of (g, u) pairs, 8 of d_h.  A thread has
// kItems of them, a CTA's width apart, so that a warp reads and writes whole
// lines, and reads them all before it writes any: d_gu may be gu.
// 512 x 8192 with a product of 64 features after it (us): 22.9 with two items,
// 23.6 with one, 23.9 with four; 25.1 where as many CTAs as are resident walked
// the items (the next item's loads waited for the last one's results).
__global__ void __launch_bounds__(kThreads) q4gsw_gated_grad_kernel(const __half* gu, const __half* d_h, __half* d_gu,
                                                                    size_t items, int act) {
  griddep_launch_dependents();
  griddep_wait();
  const size_t first = blockIdx.x * (size_t)(kThreads * kItems) + threadIdx.x;
  uint4 p[kItems];
  uint2 dh[kItems];
#pragma unroll
  for (int q = 0; q < kItems; ++q) {
    const size_t i = first + q * kThreads;
    if (i < items) {
      p[q] = reinterpret_cast<const uint4*>(gu)[i];
      dh[q] = reinterpret_cast<const uint2*>(d_h)[i];
    }
  }
#pragma unroll
  for (int q = 0; q < kItems; ++q) {
    const size_t i = first + q * kThreads;
    if (i >= items) return;
    const uint32_t pw[4] = {p[q].x, p[q].y, p[q].z, p[q].w};
    const float2 d01 = __half22float2(u32_as_h2(dh[q].x)), d23 = __half22float2(u32_as_h2(dh[q].y));
    const float d[4] = {d01.x, d01.y, d23.x, d23.y};
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = __half22float2(u32_as_h2(pw[j]));   // (g, u)
      float slope;
      const float a = act_value_slope(within(v.x), act, slope);
      out[j] = h2_as_u32(__floats2half2_rn(d[j] * within(v.y) * slope, d[j] * a));
    }
    reinterpret_cast<uint4*>(d_gu)[i] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// Threads of the projection's gradient: 8 features each, kAcross to a strip of
// STRIP features, kDown rows, ROWS of them kDown apart in flight per thread.
template <int STRIP, int ROWS>
struct Strip {
  static constexpr int kAcross = STRIP / 8, kDown = kThreads / kAcross, kGroup = kDown * ROWS;
};

// grid = (strips, C row ranges), cluster = (1, C, 1).  Thread (tx, ty) walks
// rows ty, ty + kDown, ... of its range at features 8 tx .. + 7 of the strip; the
// column sums go over a warp's rows by shuffles, over the warps in shared memory
// and over the C ranges through distributed shared memory, all in a fixed order:
// the same bits from every call, where atomics would vary.  z and d_z are null
// without an activation; d_z may be z or d_y (each element is read, then written,
// by one thread).
//
// Strips of 32 features with two rows in flight make more and shorter CTAs, and
// leave a cluster out where it only added a barrier behind the stores; strips of
// 64 with four read whole lines and have more bytes in flight.  Measured with an
// activation and d_bias, a product of 64 features after it (us, 32 and 64):
// 256 x 14336 22.2 and 24.2, 640 x 14336 37.4 and 40.3, 1021 x 14336 61 and 47.6,
// 4096 x 8192 102 and 88.9: by the number of elements (launch_act_grad).
template <int STRIP, int ROWS>
__global__ void __launch_bounds__(kThreads) q4gsw_act_grad_kernel(const __half* z, const __half* d_y, __half* d_z,
                                                                  float* __restrict__ d_bias, int M, int N, int act) {
  constexpr int kAcross = Strip<STRIP, ROWS>::kAcross, kDown = Strip<STRIP, ROWS>::kDown;
  __shared__ float part[kThreads / 32][STRIP];
  __shared__ float sums[STRIP];
  griddep_launch_dependents();
  griddep_wait();
  const int tx = threadIdx.x % kAcross, ty = threadIdx.x / kAcross;
  const int C = gridDim.y, rank = blockIdx.y;
  const int n = STRIP * blockIdx.x + 8 * tx;
  const int r_end = (int)((long long)(rank + 1) * M / C);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  if (n < N) {   // N % 8 == 0
    // rows in groups of ROWS: all loads of a group are in flight together
    for (int r0 = (int)((long long)rank * M / C) + ty; r0 < r_end; r0 += kDown * ROWS) {
      uint4 dv[ROWS], zv[ROWS];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int r = r0 + kDown * u;
        const size_t at = (size_t)(r < r_end ? r : r0) * N + n;
        dv[u] = *reinterpret_cast<const uint4*>(d_y + at);
        if (z) zv[u] = *reinterpret_cast<const uint4*>(z + at);
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int r = r0 + kDown * u;
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
            act_value_slope(within(f.x), act, s0);
            act_value_slope(within(f.y), act, s1);
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
  // over the rows of a warp (lanes kAcross apart), then over the warps
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int o = kAcross; o < 32; o *= 2) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
  }
  if ((threadIdx.x & 31) < kAcross) {
#pragma unroll
    for (int j = 0; j < 8; ++j) part[threadIdx.x >> 5][8 * tx + j] = acc[j];
  }
  __syncthreads();
  if (threadIdx.x < STRIP) {
    float s = 0.f;
    for (int y = 0; y < kThreads / 32; ++y) s += part[y][threadIdx.x];
    sums[threadIdx.x] = s;
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (C > 1) cluster.sync();
  else __syncthreads();
  if (rank == 0 && threadIdx.x < STRIP && STRIP * blockIdx.x + threadIdx.x < N) {
    float s = sums[threadIdx.x];
    for (int q = 1; q < C; ++q) s += cluster.map_shared_rank(sums, q)[threadIdx.x];
    d_bias[STRIP * blockIdx.x + threadIdx.x] = s;
  }
  if (C > 1) cluster.sync();   // no CTA leaves while rank 0 reads its sums
}

}  // namespace layer

cudaError_t launch_gated_grad(const __half* gu, const __half* d_h, int M, int F, int act, __half* d_gu,
                              cudaStream_t stream) {
  const size_t items = (size_t)M * (size_t)F / 4, per = layer::kThreads * layer::kItems;
  const size_t grid = (items + per - 1) / per;
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

template <int STRIP, int ROWS>
static cudaError_t launch_act_grad_strips(const __half* z, const __half* d_y, int M, int N, int act, __half* d_z,
                                          float* d_bias, cudaStream_t stream) {
  const int strips = (N + STRIP - 1) / STRIP;
  // row ranges: about two CTAs per SM, at least one group of rows in each
  const int sms = sm_count(current_device());
  int C = 1;
  while (C < 8 && (long long)strips * C < 2LL * sms && M / (2 * C) >= layer::Strip<STRIP, ROWS>::kGroup) C *= 2;
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
  return cudaLaunchKernelEx(&cfg, layer::q4gsw_act_grad_kernel<STRIP, ROWS>, z, d_y, d_z, d_bias, M, N, act);
}

cudaError_t launch_act_grad(const __half* z, const __half* d_y, int M, int N, int act, __half* d_z, float* d_bias,
                            cudaStream_t stream) {
  return (long long)M * N <= 10000000 ? launch_act_grad_strips<32, 2>(z, d_y, M, N, act, d_z, d_bias, stream)
                                      : launch_act_grad_strips<64, 4>(z, d_y, M, N, act, d_z, d_bias, stream);
}

}  // namespace q4gsw
