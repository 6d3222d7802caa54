// q4gsw_grads.cu - the global norm over a list of gradients, and clipping
// (sm_100a).
//
//   norm = |inv_scale| sqrt(sum g^2),  out = inv_scale min(1, max_norm / (norm + 1e-6)) g
//
// Two launches whatever the number of tensors (one for a short list).  The list is cut into pieces of 1024
// elements of one tensor, each with a record in a table in device memory,
// and every CTA has an equal run of pieces, eight in flight.  The first launch leaves
// one partial sum per CTA; the second adds them (each CTA for itself, in a fixed order,
// so no CTA waits for another) and scales, from the end of the list, whose gradients
// the L2 still holds.  A tensor that does not start on 16 bytes has its pieces counted
// from the boundary before it: all but its first and last four elements are read in
// vectors all the same.
//
// fp32 squares are taken and summed in fp64, in which no product of two fp32 values
// overflows or underflows.  fp16 squares are exact in fp32; four of them are added
// there (2^-24 of the sum each) before the fp64 sum.
//
// Norm of 201 M fp32 elements 118 us and of as many fp16 64 (the copy rate of those
// bytes: 123 and 61); 224 gradients of 11.3 M elements together 11.9, their clip into
// other buffers 23.7.  With a test per load (loads one after another) the clip takes 34
// and the norm over fp16 views that start anywhere 149 instead of 87 us.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>

#include "q4gsw_common.cuh"
#include "q4gsw_internal.h"

namespace cg = cooperative_groups;

namespace q4gsw {
namespace grads {

constexpr int kThreads = 256;
constexpr int kGroup = 4;                       // elements of a thread in a piece: whole lines a warp
constexpr int kPiece = kThreads * kGroup;
constexpr int kBatch = 8;                       // pieces in flight
constexpr int kMaxCtas = 592;                   // 4 of 148 SMs
constexpr int64_t kMaxPieces = 1 << 26;         // 2 GB of table

// What a CTA needs to know of a piece, in one load.  Both pointers count from the
// 16-byte boundary at or before the gradient's piece; `skip` elements there belong to
// nobody (the first piece of a tensor that starts off a boundary), `left` elements from
// there on reach the tensor's end (0: an unused record behind the list).
struct Piece {
  const void* grad;
  void* out;
  int64_t left;
  int32_t skip;
  int32_t halves;                 // bit 0: the gradient, bit 1: the output; bit 2: there is no output
};
static_assert(sizeof(Piece) == 32, "two loads of 16 bytes");

// Elements at + k kPiece .. + 3 of a piece and its successors for k < pieces <= kBatch,
// zero outside the tensor.  One test for the whole batch, so that its loads are issued
// together.
__device__ __forceinline__ void load_batch(const Piece& e, int at, int pieces, float (&v)[kBatch][kGroup]) {
  if (at >= e.skip && at + (pieces - 1) * kPiece + kGroup <= e.left) {
    if (e.halves & 1) {
      const uint2* p = reinterpret_cast<const uint2*>(static_cast<const __half*>(e.grad) + at);
      uint2 r[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) r[k] = k < pieces ? p[k * (kPiece / 4)] : make_uint2(0u, 0u);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float2 a = __half22float2(u32_as_h2(r[k].x)), b = __half22float2(u32_as_h2(r[k].y));
        v[k][0] = a.x, v[k][1] = a.y, v[k][2] = b.x, v[k][3] = b.y;
      }
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(e.grad) + at);
      float4 r[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) r[k] = k < pieces ? p[k * (kPiece / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) v[k][0] = r[k].x, v[k][1] = r[k].y, v[k][2] = r[k].z, v[k][3] = r[k].w;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < kBatch; ++k)
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const int j = at + k * kPiece + i;
      v[k][i] = k >= pieces || j < e.skip || j >= e.left ? 0.f
                : e.halves & 1                           ? __half2float(static_cast<const __half*>(e.grad)[j])
                                                         : static_cast<const float*>(e.grad)[j];
    }
}

// `wide`: the output is on a boundary where the gradient is
__device__ __forceinline__ void store_group(const Piece& e, bool wide, int at, const float (&v)[kGroup]) {
  if (wide && at >= e.skip && at + kGroup <= e.left) {
    if (e.halves & 2)
      *reinterpret_cast<uint2*>(static_cast<__half*>(e.out) + at) =
          make_uint2(h2_as_u32(__floats2half2_rn(v[0], v[1])), h2_as_u32(__floats2half2_rn(v[2], v[3])));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(e.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < kGroup; ++i)
    if (at + i >= e.skip && at + i < e.left) {
      if (e.halves & 2) static_cast<__half*>(e.out)[at + i] = __float2half_rn(v[i]);
      else static_cast<float*>(e.out)[at + i] = v[i];
    }
}

// Calls body(piece, pieces of its tensor up to kBatch) over this CTA's run of pieces;
// the next record is on its way meanwhile (201 M fp16 elements: 73 us without).
template <class F>
__device__ __forceinline__ void for_pieces(const Piece* table, int pieces, int run, F&& body) {
  int p = (int)((int64_t)run * pieces / gridDim.x);
  const int end = (int)((int64_t)(run + 1) * pieces / gridDim.x);
  if (p >= end) return;
  const uint4* record = reinterpret_cast<const uint4*>(table + p);
  uint4 lo = record[0], hi = record[1];
  while (p < end) {
    Piece e;
    e.grad = reinterpret_cast<const void*>((uint64_t)lo.y << 32 | lo.x);
    e.out = reinterpret_cast<void*>((uint64_t)lo.w << 32 | lo.z);
    e.left = (int64_t)((uint64_t)hi.y << 32 | hi.x);
    e.skip = (int)hi.z;
    e.halves = (int)hi.w;
    if (e.left == 0) return;             // behind the list
    const int64_t more = (e.left + kPiece - 1) / kPiece;
    int n = end - p < kBatch ? end - p : kBatch;
    n = more < n ? (int)more : n;
    p += n;
    if (p < end) {
      record = reinterpret_cast<const uint4*>(table + p);
      lo = record[0];
      hi = record[1];
    }
    body(e, n);
  }
}

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

__device__ __forceinline__ double norm_of(double squares, float inv_scale) {
  return fabs((double)inv_scale) * sqrt(squares);
}
__device__ __forceinline__ double total_norm(const double* part, int parts, float inv_scale, double* s_part) {
  double v = 0.;
  for (int i = threadIdx.x; i < parts; i += kThreads) v += part[i];
  return norm_of(cta_sum(v, s_part), inv_scale);
}

// inv_scale min(1, max_norm / (norm + 1e-6)), where min keeps a NaN and an infinite
// max_norm never clips: `first` times `second`, which is 1 but where the factor is near the
// least normal fp32 number or below (it would lose its bits there, and a large gradient
// times it is an ordinary number).
struct Factor {
  float first, second;
};
__device__ __forceinline__ Factor clip_factor(double norm, float max_norm, float inv_scale) {
  double clip = isinf(max_norm) && !isnan(norm) ? 1. : (double)max_norm / (norm + 1e-6);
  if (clip > 1.) clip = 1.;
  const double f = (double)inv_scale * clip;
  if (fabs(f) < 0x1p-100) return {(float)(f * 0x1p64), 0x1p-64f};
  return {(float)f, 1.f};
}

// This CTA's run of pieces: its sum of squares, and its outputs.
__device__ __forceinline__ double run_squares(const Piece* table, int pieces, int run) {
  double sum = 0.;
  for_pieces(table, pieces, run, [&](const Piece& e, int n) {
    float v[kBatch][kGroup];
    load_batch(e, (int)threadIdx.x * kGroup, n, v);
    if (e.halves & 1) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) s = fmaf(v[k][i], v[k][i], s);
        sum += (double)s;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < kGroup; ++i) sum = fma((double)v[k][i], (double)v[k][i], sum);
    }
  });
  return sum;
}
__device__ __forceinline__ void run_scale(const Piece* table, int pieces, int run, Factor factor) {
  for_pieces(table, pieces, run, [&](const Piece& e, int n) {
    if (e.halves & 4 || (factor.first == 1.f && e.out == e.grad && e.halves != 1 && e.halves != 2)) return;
    const bool wide = (reinterpret_cast<uintptr_t>(e.out) & (e.halves & 2 ? 7u : 15u)) == 0;
    const int at = (int)threadIdx.x * kGroup;
    float v[kBatch][kGroup];
    load_batch(e, at, n, v);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) v[k][i] = v[k][i] * factor.first * factor.second;
      if (k < n) store_group(e, wide, at + k * kPiece, v[k]);
    }
  });
}

// Few pieces: one cluster does both passes in one launch, each CTA's sum read by the
// others from its shared memory, in rank order.
template <bool CLIP>
__global__ void __launch_bounds__(kThreads)
q4gsw_grad_few_kernel(const Piece* table, int pieces, float max_norm, float inv_scale, float* norm) {
  __shared__ double s_part[kThreads / 32], s_sum;
  griddep_launch_dependents();
  griddep_wait();
  const double mine = cta_sum(run_squares(table, pieces, blockIdx.x), s_part);
  if (threadIdx.x == 0) s_sum = mine;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  double squares = 0.;
  for (int k = 0; k < (int)gridDim.x; ++k) squares += *cluster.map_shared_rank(&s_sum, k);
  const double n = norm_of(squares, inv_scale);
  if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)n;
  if (CLIP) run_scale(table, pieces, blockIdx.x, clip_factor(n, max_norm, inv_scale));
  cluster.sync();      // no CTA leaves while another reads its sum
}

__global__ void __launch_bounds__(kThreads, 4)
q4gsw_grad_squares_kernel(const Piece* table, int pieces, double* part) {
  __shared__ double s_part[kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const double sum = cta_sum(run_squares(table, pieces, blockIdx.x), s_part);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads)
q4gsw_grad_norm_kernel(const double* part, int parts, float inv_scale, float* norm) {
  __shared__ double s_part[kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const double n = total_norm(part, parts, inv_scale, s_part);
  if (threadIdx.x == 0) norm[0] = (float)n;
}

__global__ void __launch_bounds__(kThreads, 4)
q4gsw_grad_scale_kernel(const Piece* table, int pieces, const double* part, int parts, float max_norm, float inv_scale,
                        float* norm) {
  __shared__ double s_part[kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const double n = total_norm(part, parts, inv_scale, s_part);
  if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)n;
  run_scale(table, pieces, gridDim.x - 1 - blockIdx.x, clip_factor(n, max_norm, inv_scale));
}

// Up to kGradFewRecords pieces, a batch a CTA, one cluster does it: a call takes 8.3 us in place
// of 10.8 (a launch less), the GPU 6.7 in place of 6.3 (clip of 60000 elements); with twice
// as many it would take 8.1.
constexpr int kFewCtas = 8;

}  // namespace grads

// Pieces of one tensor that starts `shift` elements behind a boundary.
static int64_t grad_pieces(int64_t size, int64_t shift) {
  return size ? (size + shift + grads::kPiece - 1) / grads::kPiece : 0;
}

size_t grad_table_bytes(int count, const int64_t* sizes) {
  int64_t pieces = 0;
  for (int i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > ((int64_t)1 << 44)) return 0;
    pieces += grad_pieces(sizes[i], 7);      // the largest shift
    if (pieces > grads::kMaxPieces) return 0;
  }
  return sizeof(grads::Piece) * (size_t)(pieces ? pieces : 1);
}

void grad_table_fill(int count, const void* const* grads_in, const int* half_grads, void* const* outs,
                     const int* half_outs, const int64_t* sizes, void* table, size_t table_bytes) {
  unsigned char* t = static_cast<unsigned char*>(table);
  std::memset(t, 0, table_bytes);
  for (int i = 0; i < count; ++i) {
    const int size = half_grads[i] ? 2 : 4, out_size = outs && half_outs[i] ? 2 : 4;
    const uintptr_t grad = reinterpret_cast<uintptr_t>(grads_in[i]);
    const int64_t shift = sizes[i] ? (int64_t)(grad & 15u) / size : 0;
    const int64_t n = grad_pieces(sizes[i], shift);
    for (int64_t p = 0; p < n; ++p) {
      const int64_t first = p * grads::kPiece - shift;      // the piece's first element
      grads::Piece e;
      e.grad = reinterpret_cast<const void*>(grad + (uintptr_t)(first * size));
      e.out = outs ? reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(outs[i]) + (uintptr_t)(first * out_size)) : nullptr;
      e.left = sizes[i] - first;
      e.skip = first < 0 ? (int32_t)-first : 0;
      e.halves = (half_grads[i] ? 1 : 0) | (!outs ? 4 : half_outs[i] ? 2 : 0);
      std::memcpy(t, &e, sizeof(e));
      t += sizeof(e);
    }
  }
}

size_t grad_workspace_bytes() { return sizeof(double) * grads::kMaxCtas; }

static int grad_ctas(int pieces) { return pieces < grads::kMaxCtas ? pieces : grads::kMaxCtas; }

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

template <bool CLIP>
static cudaError_t launch_grad_few(const grads::Piece* table, int pieces, float max_norm, float inv_scale, float* norm,
                                   cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = grad_config(attr, grads::kFewCtas, stream);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = grads::kFewCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grads::q4gsw_grad_few_kernel<CLIP>, table, pieces, max_norm, inv_scale, norm);
}

cudaError_t launch_grad_norm(const void* table, size_t table_bytes, float inv_scale, float* norm, void* workspace,
                             cudaStream_t stream, char* route, int route_len) {
  const grads::Piece* t = static_cast<const grads::Piece*>(table);
  const int pieces = (int)(table_bytes / sizeof(grads::Piece)), ctas = grad_ctas(pieces);
  const bool few = pieces <= kGradFewRecords;
  snprintf(route, route_len, "grad_norm launches=%d", few ? 1 : 2);
  if (few) return launch_grad_few<false>(t, pieces, 1.f, inv_scale, norm, stream);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = grad_config(attr, ctas, stream);
  double* part = static_cast<double*>(workspace);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, grads::q4gsw_grad_squares_kernel, t, pieces, part);
  if (e != cudaSuccess) return e;
  cfg = grad_config(attr, 1, stream);
  return cudaLaunchKernelEx(&cfg, grads::q4gsw_grad_norm_kernel, (const double*)part, ctas, inv_scale, norm);
}

cudaError_t launch_grad_clip(const void* table, size_t table_bytes, float max_norm, float inv_scale, float* norm,
                             void* workspace, cudaStream_t stream, char* route, int route_len) {
  const grads::Piece* t = static_cast<const grads::Piece*>(table);
  const int pieces = (int)(table_bytes / sizeof(grads::Piece)), ctas = grad_ctas(pieces);
  const bool few = pieces <= kGradFewRecords;
  snprintf(route, route_len, "grad_clip launches=%d", few ? 1 : 2);
  if (few) return launch_grad_few<true>(t, pieces, max_norm, inv_scale, norm, stream);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = grad_config(attr, ctas, stream);
  double* part = static_cast<double*>(workspace);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, grads::q4gsw_grad_squares_kernel, t, pieces, part);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, grads::q4gsw_grad_scale_kernel, t, pieces, (const double*)part, ctas, max_norm,
                            inv_scale, norm);
}

}  // namespace q4gsw
