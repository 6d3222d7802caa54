// q4gsw_grads.cu - the global norm over a list of gradients, and clipping
// (sm_100a).
//
//   norm = |inv_scale| sqrt(sum g^2),  out = inv_scale min(1, max_norm / (norm + 1e-6)) g
//
// Two launches whatever the number of tensors.  The list is cut into pieces of 8192
// elements of one tensor; a table in device memory says for every piece whose it is.
// The first launch leaves one partial sum per CTA; the second adds them (each CTA for
// itself, in a fixed order, so no CTA waits for another) and scales its pieces.
// Squares are taken and summed in fp64, in which no product of two fp32 values
// overflows or underflows; the conversions and sums hide behind the loads.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "q4gsw_common.cuh"
#include "q4gsw_internal.h"

namespace q4gsw {
namespace grads {

constexpr int kPiece = 8192;      // elements
constexpr int kThreads = 256;
constexpr int kMaxCtas = 1184;    // 8 of 148 SMs
constexpr int kGroup = 8;         // elements of a thread's step

struct Entry {
  const void* grad;
  void* out;
  int64_t size;
  int64_t first;                  // its first piece
  int32_t half_grad, half_out;
};
struct Head {
  int64_t pieces;
  int64_t pad;
};
// Head, Entry[count], int32 tensor of each piece

__host__ __device__ inline size_t map_offset(int count) { return sizeof(Head) + sizeof(Entry) * (size_t)count; }

// 8 elements from `at` on, those past `n` zero; `wide`: the tensor starts on 16 bytes
// (every piece and group then does, 8 elements of either type at a time)
__device__ __forceinline__ void load_group(const void* p, int half, bool wide, int64_t at, int64_t n, float (&v)[kGroup]) {
  if (wide && at + kGroup <= n) {
    if (half) {
      const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const __half*>(p) + at);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(u32_as_h2(w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kGroup; ++i)
    v[i] = at + i >= n ? 0.f
           : half      ? __half2float(static_cast<const __half*>(p)[at + i])
                       : static_cast<const float*>(p)[at + i];
}

__device__ __forceinline__ void store_group(void* p, int half, bool wide, int64_t at, int64_t n, const float (&v)[kGroup]) {
  if (wide && at + kGroup <= n) {
    if (half) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = h2_as_u32(__floats2half2_rn(v[2 * i], v[2 * i + 1]));
      *reinterpret_cast<uint4*>(static_cast<__half*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
      d[0] = make_float4(v[0], v[1], v[2], v[3]);
      d[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kGroup; ++i)
    if (at + i < n) {
      if (half) static_cast<__half*>(p)[at + i] = __float2half_rn(v[i]);
      else static_cast<float*>(p)[at + i] = v[i];
    }
}

__device__ __forceinline__ bool wide16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The sum of `v` over the CTA, in a fixed order, in every thread.
__device__ __forceinline__ double cta_sum(double v, double* s_part) {
#pragma unroll
  for (int o = 16; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) s_part[threadIdx.x / 32] = v;
  __syncthreads();
  double s = 0.;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += s_part[w];
  return s;
}

__global__ void __launch_bounds__(kThreads)
q4gsw_grad_squares_kernel(const unsigned char* table, int count, double* part) {
  __shared__ double s_part[kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t pieces = reinterpret_cast<const Head*>(table)->pieces;
  const Entry* entries = reinterpret_cast<const Entry*>(table + sizeof(Head));
  const int32_t* owner = reinterpret_cast<const int32_t*>(table + map_offset(count));
  double sum = 0.;
  for (int64_t p = blockIdx.x; p < pieces; p += gridDim.x) {
    const Entry e = entries[owner[p]];
    const bool wide = wide16(e.grad);
    const int64_t at = (p - e.first) * kPiece;
#pragma unroll
    for (int k = 0; k < kPiece / (kThreads * kGroup); ++k) {
      float v[kGroup];
      load_group(e.grad, e.half_grad, wide, at + (k * kThreads + (int)threadIdx.x) * kGroup, e.size, v);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) sum = fma((double)v[i], (double)v[i], sum);
    }
  }
  sum = cta_sum(sum, s_part);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ float total_norm(const double* part, int parts, float inv_scale, double* s_part) {
  double v = 0.;
  for (int i = threadIdx.x; i < parts; i += kThreads) v += part[i];
  return (float)(fabs((double)inv_scale) * sqrt(cta_sum(v, s_part)));
}

__global__ void __launch_bounds__(kThreads)
q4gsw_grad_norm_kernel(const double* part, int parts, float inv_scale, float* norm) {
  __shared__ double s_part[kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const float n = total_norm(part, parts, inv_scale, s_part);
  if (threadIdx.x == 0) norm[0] = n;
}

__global__ void __launch_bounds__(kThreads)
q4gsw_grad_scale_kernel(const unsigned char* table, int count, const double* part, int parts,
                        float max_norm, float inv_scale, float* norm) {
  __shared__ double s_part[kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const float n = total_norm(part, parts, inv_scale, s_part);
  if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = n;
  // min(1, .) that keeps a NaN; an infinite max_norm never clips
  float clip = isinf(max_norm) && !isnan(n) ? 1.f : max_norm / (n + 1e-6f);
  if (clip > 1.f) clip = 1.f;
  const float factor = inv_scale * clip;
  const int64_t pieces = reinterpret_cast<const Head*>(table)->pieces;
  const Entry* entries = reinterpret_cast<const Entry*>(table + sizeof(Head));
  const int32_t* owner = reinterpret_cast<const int32_t*>(table + map_offset(count));
  for (int64_t p = blockIdx.x; p < pieces; p += gridDim.x) {
    const Entry e = entries[owner[p]];
    if (factor == 1.f && e.out == e.grad && e.half_out == e.half_grad) continue;
    const bool wide = wide16(e.grad), wide_out = wide16(e.out);
    const int64_t at = (p - e.first) * kPiece;
    constexpr int kSteps = kPiece / (kThreads * kGroup);
    float v[kSteps][kGroup];
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
      load_group(e.grad, e.half_grad, wide, at + (k * kThreads + (int)threadIdx.x) * kGroup, e.size, v[k]);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) v[k][i] *= factor;
      store_group(e.out, e.half_out, wide_out, at + (k * kThreads + (int)threadIdx.x) * kGroup, e.size, v[k]);
    }
  }
}

}  // namespace grads

size_t grad_table_bytes(int count, const int64_t* sizes) {
  int64_t pieces = 0;
  for (int i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > ((int64_t)1 << 44)) return 0;
    pieces += (sizes[i] + grads::kPiece - 1) / grads::kPiece;
    if (pieces > 0x7fffffff) return 0;
  }
  return round_up(grads::map_offset(count) + sizeof(int32_t) * (size_t)pieces, 16);
}

size_t grad_table_least(int count) { return round_up(grads::map_offset(count), 16); }

void grad_table_fill(int count, const void* const* grads_in, const int* half_grads, void* const* outs,
                     const int* half_outs, const int64_t* sizes, void* table) {
  unsigned char* t = static_cast<unsigned char*>(table);
  int64_t pieces = 0;
  for (int i = 0; i < count; ++i) {
    grads::Entry e;
    std::memset(&e, 0, sizeof(e));
    e.grad = grads_in[i];
    e.out = outs ? outs[i] : nullptr;
    e.size = sizes[i];
    e.first = pieces;
    e.half_grad = half_grads[i];
    e.half_out = outs ? half_outs[i] : 0;
    std::memcpy(t + sizeof(grads::Head) + sizeof(e) * (size_t)i, &e, sizeof(e));
    const int64_t n = (sizes[i] + grads::kPiece - 1) / grads::kPiece;
    for (int64_t p = 0; p < n; ++p) {
      const int32_t who = i;
      std::memcpy(t + grads::map_offset(count) + sizeof(int32_t) * (size_t)(pieces + p), &who, sizeof(who));
    }
    pieces += n;
  }
  grads::Head h{pieces, 0};
  std::memcpy(t, &h, sizeof(h));
}

size_t grad_workspace_bytes() { return sizeof(double) * grads::kMaxCtas; }

static int grad_ctas(size_t table_bytes, int count) {
  // the map is padded by at most three words: no CTA too few
  const size_t most = (table_bytes - grads::map_offset(count)) / sizeof(int32_t);
  return most < 1 ? 1 : most < (size_t)grads::kMaxCtas ? (int)most : grads::kMaxCtas;
}

static cudaLaunchConfig_t grad_config(cudaLaunchAttribute* attr, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(grads::kThreads, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

cudaError_t launch_grad_norm(const void* table, size_t table_bytes, int count, float inv_scale, float* norm,
                             void* workspace, cudaStream_t stream) {
  const int ctas = grad_ctas(table_bytes, count);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = grad_config(attr, ctas, stream);
  double* part = static_cast<double*>(workspace);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, grads::q4gsw_grad_squares_kernel,
                                           static_cast<const unsigned char*>(table), count, part);
  if (e != cudaSuccess) return e;
  cfg = grad_config(attr, 1, stream);
  return cudaLaunchKernelEx(&cfg, grads::q4gsw_grad_norm_kernel, (const double*)part, ctas, inv_scale, norm);
}

cudaError_t launch_grad_clip(const void* table, size_t table_bytes, int count, float max_norm, float inv_scale,
                             float* norm, void* workspace, cudaStream_t stream) {
  const int ctas = grad_ctas(table_bytes, count);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = grad_config(attr, ctas, stream);
  double* part = static_cast<double*>(workspace);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, grads::q4gsw_grad_squares_kernel,
                                           static_cast<const unsigned char*>(table), count, part);
  if (e != cudaSuccess) return e;
  cfg = grad_config(attr, ctas, stream);
  return cudaLaunchKernelEx(&cfg, grads::q4gsw_grad_scale_kernel, static_cast<const unsigned char*>(table), count,
                            (const double*)part, ctas, max_norm, inv_scale, norm);
}

}  // namespace q4gsw
