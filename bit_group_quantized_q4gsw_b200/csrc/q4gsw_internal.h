// q4gsw_internal.h - launchers shared between the translation units of the
// library.  Not part of the C ABI.
#pragma once

#include <atomic>
#include <cstdint>
#include <mutex>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace q4gsw {

// Token counts up to this run the tensor-core GEMV (weight streaming); above
// it the tcgen05 GEMM.
constexpr int kGemvMaxM = 16;

// Route pins of the calling host thread (set by q4gsw_debug_pin_routes; 0
// everywhere means the launchers choose).  Thread-local, like the route string.
enum GemvPin { kGemvAuto = 0, kGemvReg = 1, kGemvTma = 2, kGemvTmaXs = 3 };
enum GemmPin { kGemmAuto = 0, kGemmTs = 1, kGemmSs = 2, kGemmSs1 = 3, kGemmSs2 = 4 };
struct RoutePins {
  int gemv = kGemvAuto;
  int gemm = kGemmAuto;
};
RoutePins& route_pins();

// One-time set-up per device (cudaFuncSetAttribute of one kernel variant),
// safe when several host threads make their first call at the same time: the
// first caller runs `fn`, the others wait for it and then see its result.
constexpr int kMaxDevices = 64;
struct PerDeviceOnce {
  std::once_flag flag[kMaxDevices];
  std::atomic<int> err[kMaxDevices];
};
template <typename F>
inline cudaError_t once_per_device(PerDeviceOnce& o, int dev, F&& fn) {
  if (dev < 0 || dev >= kMaxDevices) return fn();   // not cached
  std::call_once(o.flag[dev], [&] { o.err[dev].store(static_cast<int>(fn())); });
  return static_cast<cudaError_t>(o.err[dev].load());
}

// Device the calling thread is bound to (cudaGetDevice), and its SM count.
int current_device();
int sm_count(int dev);

// f32s: the blob holds fp32 scales (packed layout version 2) instead of fp16.
cudaError_t launch_prepack(const uint8_t* codes, const void* scales, int N, int K, int gs, bool f32s, void* packed,
                           cudaStream_t stream, uint32_t* host_flag);
// The gated block's blob: N = 2 F rows, gate row j and up row j as rows 2 j and 2 j + 1.
cudaError_t launch_prepack_gated(const uint8_t* codes_gate, const void* scales_gate, const uint8_t* codes_up,
                                 const void* scales_up, int F, int K, int gs, bool f32s, void* packed,
                                 cudaStream_t stream, uint32_t* host_flag);
cudaError_t launch_unpack(const void* packed, int N, int K, uint8_t* codes, cudaStream_t stream);
cudaError_t launch_dequant(const void* packed, int N, int K, int gs, bool f32s, float* w32, uint16_t* w16,
                           cudaStream_t stream);

// Output columns [0, N) of a forward split over up to three row-major
// buffers: n < n1 -> y0[m, n], n < n2 -> y1[m, n - n1], else y2[m, n - n2]
// (the fused Q/K/V projection writes three distinct outputs).
struct OutSplit {
  float* y0;
  float* y1;
  float* y2;
  int n1, n2, N;
};

__host__ __device__ inline OutSplit single_output(float* y, int N) { return OutSplit{y, y, y, N, N, N}; }

// fp16 outputs with an epilogue (q4gsw_epilogue.cuh) over N output columns:
//   gated   v = (g, u) pairs (weight rows interleaved): y[m, j] = act(g_j) u_j,
//           z[m, 2 j] = g_j, z[m, 2 j + 1] = u_j
//   else    z[m, n] = v + bias[n],  y[m, n] = act(z) + res[m, n]
// bias, res and z may be null; y may be res.
enum ActKind { kActNone = 0, kActSilu = 1, kActGelu = 2 };
struct Epi {
  __half* y;
  __half* z;
  const __half* bias;
  const __half* res;
  int N;
  int act;
  int gated;
};

// The same of a product with an adapter for every token (q4gsw_lowrank.cuh):
//   y[m, n] = v + scale[a] sum_j inter[m, j] P_a(n, j) + bias[n] + res[m, n]
// for the tokens with an adapter a in the plan.  mat: [L, N, r], or [L, r, N] for the
// input gradient; scale may be null.  The product's activations were complete before it
// could start (griddep_wait), so they are read at once, and only the epilogue waits for
// the kernel in front, behind which inter has been written.
struct EpiLow {
  __half* y;
  const __half* bias;
  const __half* res;
  int N;
  const float* inter;
  const __half* mat;
  const float* scale;
  const int32_t* plan;
  int M, L, r;
};

// The compute launchers take f32s = the packed blob has fp32 scales (layout
// version 2) instead of fp16 (version 1).
// Tensor-core GEMV routes for small token counts.  `M` may exceed 16: token
// chunks of 16 then run as grid z-slices (each re-reads the weight).
cudaError_t launch_gemv_fwd(const void* packed, int N, int K, int gs, bool f32s, const uint16_t* x, int M,
                            OutSplit out, cudaStream_t stream, char* route, int route_len);
cudaError_t launch_gemv_bwd(const void* packed, int N, int K, int gs, bool f32s, const uint16_t* d_out, int M,
                            float* d_x, cudaStream_t stream, char* route, int route_len);

// The same products with fp16 outputs through an epilogue: any M >= 1, the
// GEMV up to kGemvMaxM tokens, the GEMMs above.
cudaError_t launch_product_low(bool bwd, const void* packed, int N, int K, int gs, bool f32s, const uint16_t* act,
                               int M, const EpiLow& out, cudaStream_t stream, char* route, int route_len);
cudaError_t launch_product_epi(bool bwd, const void* packed, int N, int K, int gs, bool f32s, const uint16_t* act,
                               int M, const Epi& out, cudaStream_t stream, char* route, int route_len);

// Forward GEMV that streams the packed weight through a TMA ring (M <= 16
// per z-slice).
cudaError_t launch_gemv_tma_fwd(const void* packed, int N, int K, int gs, bool f32s, const uint16_t* x, int M, OutSplit out,
                                cudaStream_t stream, char* route, int route_len);
cudaError_t launch_gemv_tma_bwd(const void* packed, int N, int K, int gs, bool f32s, const uint16_t* d_out, int M, float* d_x,
                                cudaStream_t stream, char* route, int route_len);

// tcgen05 GEMM routes (any M >= 1; used above the GEMV range).
cudaError_t launch_gemm_fwd(const void* packed, int N, int K, int gs, bool f32s, const uint16_t* x, int M, OutSplit out,
                            cudaStream_t stream, char* route, int route_len);
cudaError_t launch_gemm_bwd(const void* packed, int N, int K, int gs, bool f32s, const uint16_t* d_out, int M, float* d_x,
                            cudaStream_t stream, char* route, int route_len);

// Frozen-base low-rank adapter: the fp16 adapter matrix (forward B [N, r],
// backward A [r, K]), its rank (8 <= r <= 64, r % 8 == 0) and the fp16
// intermediate [M][64] (forward x A^T, backward d_out B; columns r..63 zero).
struct AdapterRef {
  const uint16_t* mat;
  int r;
  const void* inter;
};
// The intermediate: act [M][C] times the projection (by_rows: A [r, C], used
// as A^T; else B [C, r]) into `workspace` as [M][64] fp16.
cudaError_t launch_adapter_proj(const uint16_t* act, const uint16_t* proj, bool by_rows, int M, int C, int r,
                                void* workspace, cudaStream_t stream);
// Device address (on the current device) and size of the library's own fixed
// scratch array for the allocation-free adapter entry point.  The first call
// on a device looks the address up (cudaGetSymbolAddress).
constexpr size_t kNoAllocScratchBytes = (size_t)1 << 20;
cudaError_t noalloc_scratch(void** ptr, size_t* bytes);
// The tensor-memory GEMM (forward when !bwd) with the adapter stage added to
// the accumulator of the last contraction split.
cudaError_t launch_gemm_adapter(bool bwd, const void* packed, int N, int K, int gs, const uint16_t* act, int M,
                                float* out, const AdapterRef& ad, cudaStream_t stream, char* route, int route_len);

// int8 dynamically quantised activations (linear_dq8ca_q4gsw): workspace map
// (q int8 [M][K], a_s fp32 [M], a_z int32 [M]), the quantiser and the product.
size_t dq8ca_workspace_bytes(int M, int K);
size_t dq8ca_scale_offset(int M, int K);
size_t dq8ca_zero_offset(int M, int K);
cudaError_t launch_dq8ca_quantize(const uint16_t* x, int M, int K, void* workspace, cudaStream_t stream);
cudaError_t launch_dq8ca_gemv(const void* packed, int N, int K, int gs, int M, const void* workspace, OutSplit out,
                              cudaStream_t stream, char* route, int route_len);

// Gradients through the activations (q4gsw_layer.cu): d_gu from gu and d_h
// (fp16, [M][2 F] and [M][F]); d_z = d_y act'(z) and its column sums (fp16
// [M][N]; z and d_z null without an activation, d_bias may be null).
cudaError_t launch_gated_grad(const __half* gu, const __half* d_h, int M, int F, int act, __half* d_gu,
                              cudaStream_t stream);
cudaError_t launch_act_grad(const __half* z, const __half* d_y, int M, int N, int act, __half* d_z, float* d_bias,
                            cudaStream_t stream);

// Distillation loss, log-sum-exp and gradient (q4gsw_distill.cuh).
struct DistillArgs {
  const void* logits;
  const int32_t* indices;
  const void* teacher;
  const float* d_loss;    // null: no gradient
  const float* lse_in;    // backward only: the forward's log-sum-exp
  float* loss;
  float* lse;
  __half* grad;
  int M, V, k;
  int half_teacher;
  float temperature;
  float inv_t;            // 1 / temperature
};
cudaError_t launch_distill_rows(const DistillArgs& a, bool half_logits, cudaStream_t stream, char* route,
                                int route_len);
cudaError_t launch_distill_bwd(const DistillArgs& a, bool half_logits, cudaStream_t stream, char* route,
                               int route_len);

// The device error word (bits of q4gsw_device_error_check) of the current device.
cudaError_t device_error_word(unsigned int** word);

// Adapters of many requests (q4gsw_adapters.cu; the plan: q4gsw_adapters.cuh).
// down: out fp32 [M][r] = (scale) act P, the adapters' matrices [r, C] (by_rows: A) or
// [C, r] (B), by one kernel for few tiles (adapters_few) and another for many;
// grad: d_a = sums over each adapter's tokens of v^T x, d_b of scale d_y^T u, fp32.
struct AdaptersRef {
  const int32_t* plan;
  int L, r;
};
constexpr int kMaxAdapterFeatures = 64 * 65535;
cudaError_t launch_adapters_plan(const int32_t* ids, int M, int L, void* plan, cudaStream_t stream);
cudaError_t launch_adapters_down(const AdaptersRef& ad, const uint16_t* act, bool by_rows, const uint16_t* proj,
                                 const float* scale, int M, int C, float* out, cudaStream_t stream);
bool adapters_few(const AdaptersRef& ad, int M);
cudaError_t launch_adapters_grad(const AdaptersRef& ad, const uint16_t* x, const float* v, float* d_a, int K,
                                 const uint16_t* d_y, const float* u, const float* scale, float* d_b, int N, int M,
                                 bool accumulate, cudaStream_t stream);

// The norms around a block (q4gsw_norms.cu).  Pointers as in q4gsw_norms_fwd / _bwd.
struct NormsArgs {
  const __half* h;        // forward: the stream; backward: the stream after the block
  const __half* block;
  const __half* w_post;
  const __half* gate;
  const __half* w_pre;
  const __half* d_x;
  const __half* d_h;
  __half* h_out;          // forward; backward: d_residual
  __half* x;              // forward; backward: d_block
  __half* d_gate_rows;
  float* d_w_pre;
  float* d_w_post;
  float* d_gate;
  float* part;            // backward with sums over the rows: the workspace
  float residual_scale, weight_offset, eps;
  int gate_rows, M, D;
};
constexpr int kMaxNormFeatures = 32768, kMaxNormRows = 1 << 30;
size_t norms_workspace_bytes(int M, int D);
cudaError_t launch_norms_fwd(const NormsArgs& a, cudaStream_t stream, char* route, int route_len);
cudaError_t launch_norms_bwd(const NormsArgs& a, cudaStream_t stream, char* route, int route_len);

// Gradient lists (q4gsw_grads.cu): the table's bytes (0: too many pieces), its host
// contents, and the two calls.
size_t grad_table_bytes(int count, const int64_t* sizes);
void grad_table_fill(int count, const void* const* grads, const int* half_grads, void* const* outs,
                     const int* half_outs, const int64_t* sizes, void* table, size_t table_bytes);
size_t grad_workspace_bytes();
constexpr size_t kGradRecordBytes = 32;
constexpr int kGradFewRecords = 64;      // up to here one launch, without a workspace
cudaError_t launch_grad_norm(const void* table, size_t table_bytes, float inv_scale, float* norm, void* workspace,
                             cudaStream_t stream, char* route, int route_len);
cudaError_t launch_grad_clip(const void* table, size_t table_bytes, float max_norm, float inv_scale, float* norm,
                             void* workspace, cudaStream_t stream, char* route, int route_len);

// Embedding rows out[t] = dequant(W)[indices[t]] (fp32); an index outside
// [0, N) gives a zero row and sets kIndexErrorBit in the device error word.
cudaError_t launch_embedding(const void* packed, int N, int K, int gs, bool f32s, const int32_t* indices, int T, float* out,
                             cudaStream_t stream);

// One thread block that waits on a barrier nothing completes until its
// bounded wait (limit_us microseconds) runs out and records a time-out.
cudaError_t launch_wait_probe(unsigned int limit_us, cudaStream_t stream);

// Swaps the device word in which kernels record waits that ran out (and
// embedding indices out of range) with 0 in one atomic operation, ordered on
// `stream`, and returns the old value; synchronises `stream`.
cudaError_t read_and_clear_device_error(cudaStream_t stream, unsigned int* host_value);

}  // namespace q4gsw
