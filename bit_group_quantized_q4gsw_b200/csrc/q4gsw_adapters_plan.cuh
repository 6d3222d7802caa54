// q4gsw_adapters_plan.cuh - the tokens of a batch in the order of their
// adapters (sm_100a).  Included once, by q4gsw_gemm_sm100.cu, which owns the
// device error word.
//
// A stable counting sort in one CTA.  The 32 warps own consecutive ranges of the
// tokens; each counts its adapters in a histogram of its own (the lanes of equal
// ids are found by a match, so that no two lanes add to one counter), the
// histograms are summed over (adapter, warp) in that order, and each warp walks its
// range again and places its tokens.  Nothing is decided by the order of atomics:
// tokens of one adapter keep their order, and sums over them are the same in
// every call.  It runs once a batch, on one SM: M = 4096 are four rounds of 32 tokens a
// warp, and a long prompt pays one SM's rate (us, M and L): 5.7 (1, 4), 5.9 (16, 32),
// 6.8 (512, 8), 12.2 (4096, 16), 19.4 (4096, 1024), 147 and 276 (100000, 16 and 1024),
// 2103 (1000000, 64).
#pragma once

#include "q4gsw_adapters.cuh"

namespace q4gsw {
namespace ma {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// groups 0 .. L - 1 are the adapters, group L the tokens without one
__device__ __forceinline__ int plan_group(int id, int L) { return id >= 0 && id < L ? id : L; }

__global__ void __launch_bounds__(kPlanThreads)
q4gsw_adapters_plan_kernel(const int32_t* ids, int M, int L, int32_t* plan) {
  extern __shared__ int s_hist[];          // [kPlanWarps][G], then the tiles before each group [G + 1]
  __shared__ int s_sum[3][kPlanWarps];
  griddep_launch_dependents();
  griddep_wait();
  const PlanView P = plan_view(plan, M, L);
  const int G = L + 1;
  int* s_tile = s_hist + kPlanWarps * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * G; i += kPlanThreads) s_hist[i] = 0;
  __syncthreads();
  const int begin = (int)((long long)warp * M / kPlanWarps), end = (int)((long long)(warp + 1) * M / kPlanWarps);
  int* mine = s_hist + warp * G;
  bool bad = false;
  for (int m0 = begin; m0 < end; m0 += 32) {
    const int m = m0 + lane;
    int grp = -1;
    if (m < end) {
      const int id = ids[m];
      bad |= id < -1 || id >= L;
      grp = plan_group(id, L);
    }
    const unsigned same = __match_any_sync(0xffffffffu, grp);
    if (grp >= 0 && lane == __ffs(same) - 1) mine[grp] += __popc(same);
    __syncwarp();
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&g_device_error, kIndexErrorBit);
  __syncthreads();
  // thread g: group g (G <= 1025: the last group, of the tokens without an adapter, is
  // known from the others)
  int count = 0;
  if (threadIdx.x < L)
    for (int w = 0; w < kPlanWarps; ++w) count += s_hist[w * G + threadIdx.x];
  const int tiles = (count + kTileRows - 1) / kTileRows;
  const int pairs = (tiles + 1) / 2;
  // inclusive scans of counts, tiles and pairs over the threads
  int c = count, t = tiles, d = pairs;
  for (int o = 1; o < 32; o *= 2) {
    const int cu = __shfl_up_sync(0xffffffffu, c, o), tu = __shfl_up_sync(0xffffffffu, t, o),
              du = __shfl_up_sync(0xffffffffu, d, o);
    if (lane >= o) {
      c += cu;
      t += tu;
      d += du;
    }
  }
  if (lane == 31) {
    s_sum[0][warp] = c;
    s_sum[1][warp] = t;
    s_sum[2][warp] = d;
  }
  __syncthreads();
  int all_c = 0, all_t = 0, all_d = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w == warp) {
      c += all_c;
      t += all_t;
      d += all_d;
    }
    all_c += s_sum[0][w];
    all_t += s_sum[1][w];
    all_d += s_sum[2][w];
  }
  if (threadIdx.x < L) {
    P.first[threadIdx.x] = c - count;
    s_tile[threadIdx.x] = t - tiles;
    int at = c - count;      // where each warp's tokens of this group start
    for (int w = 0; w < kPlanWarps; ++w) {
      const int n = s_hist[w * G + threadIdx.x];
      s_hist[w * G + threadIdx.x] = at;
      at += n;
    }
  }
  const int none_tiles = (M - all_c + kTileRows - 1) / kTileRows;
  if (threadIdx.x == 0) {
    P.first[L] = all_c;
    P.first[L + 1] = M;
    P.head[0] = all_t + none_tiles;
    P.head[1] = M;
    P.head[2] = L;
    P.head[3] = kPlanMark;
    s_tile[L] = all_t;
    int at = all_c;
    for (int w = 0; w < kPlanWarps; ++w) {
      const int n = s_hist[w * G + L];
      s_hist[w * G + L] = at;
      at += n;
    }
  }
  // the tiles' adapters and empty rows; slots past the last tile are marked unused
  const int slots = plan_slots(M, L);
  for (int i = threadIdx.x; i < slots; i += kPlanThreads) P.tile[i] = kNoTile;
  for (int i = threadIdx.x; i < slots * kTileRows; i += kPlanThreads) P.rows[i] = -1;
  for (int i = threadIdx.x; i < plan_pairs(M, L); i += kPlanThreads) P.pair[i] = -1;
  __syncthreads();
  if (threadIdx.x < L) {
    for (int i = 0; i < tiles; ++i) P.tile[t - tiles + i] = threadIdx.x;
    for (int i = 0; i < pairs; ++i) P.pair[d - pairs + i] = t - tiles + 2 * i;
  }
  for (int i = threadIdx.x; i < none_tiles; i += kPlanThreads) P.tile[all_t + i] = kNoAdapter;
  for (int i = threadIdx.x; i < (none_tiles + 1) / 2; i += kPlanThreads) P.pair[all_d + i] = all_t + 2 * i;
  // place the tokens: in the sorted order, and in the 16 rows of their group's tiles
  for (int m0 = begin; m0 < end; m0 += 32) {
    const int m = m0 + lane;
    const int grp = m < end ? plan_group(ids[m], L) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, grp);
    int base = 0;
    if (grp >= 0) base = mine[grp];
    __syncwarp();
    if (grp >= 0) {
      const int pos = base + __popc(same & ((1u << lane) - 1u));
      if (lane == __ffs(same) - 1) mine[grp] = base + __popc(same);
      const int start = grp < L ? P.first[grp] : all_c;
      P.order[pos] = m;
      P.rows[s_tile[grp] * kTileRows + (pos - start)] = m;
    }
    __syncwarp();
  }
}

}  // namespace ma

// Address of the device error word on the current device, for kernels of other files.
cudaError_t device_error_word(unsigned int** word) {
  static PerDeviceOnce once;
  static void* address[kMaxDevices];
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  const cudaError_t e = once_per_device(once, dev, [&] { return cudaGetSymbolAddress(&address[dev], g_device_error); });
  *word = static_cast<unsigned int*>(address[dev]);
  return e;
}

cudaError_t launch_adapters_plan(const int32_t* ids, int M, int L, void* plan, cudaStream_t stream) {
  const size_t smem = sizeof(int) * ((size_t)(ma::kPlanWarps + 1) * (L + 1));   // at most 135300 bytes
  const int dev = current_device();
  static PerDeviceOnce once;
  const cudaError_t e = once_per_device(once, dev, [] {
    return cudaFuncSetAttribute(ma::q4gsw_adapters_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(sizeof(int) * (ma::kPlanWarps + 1) * (ma::kMaxAdapters + 1)));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(ma::kPlanThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ma::q4gsw_adapters_plan_kernel, ids, M, L, static_cast<int32_t*>(plan));
}

}  // namespace q4gsw
