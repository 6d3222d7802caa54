// q4gsw_adapters_api.cu - the extern "C" entry points declared in
// include/q4gsw_adapters.h: argument checks, route strings and launches.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>

#include "../../include/q4gsw_adapters.h"
#include "q4gsw_adapters.cuh"
#include "q4gsw_api_common.h"
#include "q4gsw_common.cuh"
#include "q4gsw_internal.h"

using namespace q4gsw;

namespace {

// No C++ exception may cross the C boundary.
template <typename F>
q4gsw_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return Q4GSW_ERR_CUDA;
  }
}

const __half* h(const uint16_t* p) { return reinterpret_cast<const __half*>(p); }
__half* h(uint16_t* p) { return reinterpret_cast<__half*>(p); }
bool word(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

q4gsw_status check_plan(int M, int L) {
  if (M < 0 || M > ma::kMaxPlanTokens || L < 1 || L > ma::kMaxAdapters) return Q4GSW_ERR_SHAPE;
  return Q4GSW_OK;
}

q4gsw_status check_adapters(int N, int K, int gs, int L, int r, int M) {
  const q4gsw_status st = check_weight_shape(N, K, gs);
  if (st != Q4GSW_OK) return st;
  if (N > kMaxAdapterFeatures || K > kMaxAdapterFeatures) return Q4GSW_ERR_SHAPE;
  if (r < 8 || r > 64 || r % 8) return Q4GSW_ERR_SHAPE;
  return check_plan(M, L);
}

q4gsw_status adapters_fwd_impl(const void* packed, int N, int K, int gs, bool f32s, const void* plan,
                               const uint16_t* a, const uint16_t* b, const float* scale, int L, int r,
                               const uint16_t* x, int M, const uint16_t* bias, const uint16_t* residual, uint16_t* y,
                               float* u, q4gsw_stream_t stream) {
  const q4gsw_status st = check_adapters(N, K, gs, L, r, M);
  if (st != Q4GSW_OK) return st;
  if (M == 0) {
    set_route("empty");
    return Q4GSW_OK;
  }
  if (!packed || !plan || !a || !b || !x || !y || !u) return Q4GSW_ERR_NULL;
  if (!aligned16(packed) || !aligned16(plan) || !aligned16(a) || !aligned16(b) || !aligned16(x) || !aligned16(bias) ||
      !aligned16(residual) || !aligned16(y) || !aligned16(u) || !word(scale))
    return Q4GSW_ERR_ALIGN;
  if (y == x) return Q4GSW_ERR_UNSUPPORTED;      // tiles of y are written while others are computed from x
  const AdaptersRef ad{static_cast<const int32_t*>(plan), L, r};
  cudaError_t e = launch_adapters_down(ad, x, true, a, nullptr, M, K, u, stream);
  char inner[128] = "", route[160];
  if (e == cudaSuccess) {
    const EpiLow out{h(y), h(bias), h(residual), N, u, h(b), scale, ad.plan, M, L, r};   // its epilogue adds the term
    e = launch_product_low(false, packed, N, K, gs, f32s, x, M, out, stream, inner, sizeof(inner));
  }
  snprintf(route, sizeof(route), "adapters %s launches=1 + %s", adapters_few(ad, M) ? "few" : "down", inner);
  set_route(route);
  return from_cuda(e);
}

q4gsw_status adapters_bwd_impl(const void* packed, int N, int K, int gs, bool f32s, const void* plan,
                               const uint16_t* a, const uint16_t* b, const float* scale, int L, int r,
                               const uint16_t* x, const float* u, const uint16_t* d_y, int M, int accumulate, float* v,
                               uint16_t* d_x, float* d_a, float* d_b, q4gsw_stream_t stream) {
  const q4gsw_status st = check_adapters(N, K, gs, L, r, M);
  if (st != Q4GSW_OK) return st;
  const bool grads = d_a && d_b;
  if ((!d_a) != (!d_b) || (!d_x && !grads)) return Q4GSW_ERR_NULL;
  if (!aligned16(d_a) || !aligned16(d_b)) return Q4GSW_ERR_ALIGN;
  if (M == 0) {
    set_route("empty");
    if (!grads || accumulate) return Q4GSW_OK;
    const size_t row = sizeof(float) * (size_t)L * r;
    cudaError_t e = cudaMemsetAsync(d_a, 0, row * K, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(d_b, 0, row * N, stream);
    return from_cuda(e);
  }
  if (!plan || !b || !d_y || !v || (d_x && (!packed || !a)) || (grads && (!x || !u))) return Q4GSW_ERR_NULL;
  if (!aligned16(packed) || !aligned16(plan) || !aligned16(a) || !aligned16(b) || !aligned16(x) || !aligned16(u) ||
      !aligned16(d_y) || !aligned16(v) || !aligned16(d_x) || !word(scale))
    return Q4GSW_ERR_ALIGN;
  // tiles of d_x are written while others are computed from d_y; v is there before the gradients read u
  if (d_x == d_y || (grads && ((d_x && d_x == x) || v == u))) return Q4GSW_ERR_UNSUPPORTED;
  const AdaptersRef ad{static_cast<const int32_t*>(plan), L, r};
  char inner[128] = "", route[160];
  cudaError_t e = launch_adapters_down(ad, d_y, false, b, scale, M, N, v, stream);
  if (e == cudaSuccess && grads)
    e = launch_adapters_grad(ad, x, v, d_a, K, d_y, u, scale, d_b, N, M, accumulate != 0, stream);
  if (e == cudaSuccess && d_x) {
    const EpiLow out{h(d_x), nullptr, nullptr, K, v, h(a), nullptr, ad.plan, M, L, r};
    e = launch_product_low(true, packed, N, K, gs, f32s, d_y, M, out, stream, inner, sizeof(inner));
  }
  snprintf(route, sizeof(route), "adapters %s launches=1%s%s%s", adapters_few(ad, M) ? "few" : "down",
           grads ? " + grad launches=1" : "", d_x ? " + " : "", inner);
  set_route(route);
  return from_cuda(e);
}

q4gsw_status check_norms(int M, int D, float residual_scale, float weight_offset, float eps) {
  if (M < 0 || M > kMaxNormRows || D <= 0 || D % 4 || D > kMaxNormFeatures) return Q4GSW_ERR_SHAPE;
  if (D % 8) return Q4GSW_ERR_ALIGN;   // 16-byte vectors
  if (!std::isfinite(residual_scale) || !std::isfinite(weight_offset) || !std::isfinite(eps) || eps < 0.f)
    return Q4GSW_ERR_SHAPE;
  return Q4GSW_OK;
}

}  // namespace

extern "C" {

size_t q4gsw_adapters_plan_bytes(int M, int L) {
  return check_plan(M, L) == Q4GSW_OK ? sizeof(int32_t) * ma::plan_words(M, L) : 0;
}

q4gsw_status q4gsw_adapters_plan(const int32_t* ids, int M, int L, void* plan, size_t plan_bytes,
                                 q4gsw_stream_t stream) {
  return guarded([&]() -> q4gsw_status {
    const q4gsw_status st = check_plan(M, L);
    if (st != Q4GSW_OK) return st;
    if (M == 0) {
      set_route("empty");
      return Q4GSW_OK;
    }
    if (!ids || !plan) return Q4GSW_ERR_NULL;
    if (!word(ids) || !aligned16(plan)) return Q4GSW_ERR_ALIGN;
    if (plan_bytes < sizeof(int32_t) * ma::plan_words(M, L)) return Q4GSW_ERR_SIZE;
    set_route("adapters_plan launches=1");
    return from_cuda(launch_adapters_plan(ids, M, L, plan, stream));
  });
}

q4gsw_status q4gsw_adapters_fwd(const void* packed, int N, int K, int group_size, const void* plan, const uint16_t* a,
                                const uint16_t* b, const float* scale, int L, int r, const uint16_t* x, int M,
                                const uint16_t* bias, const uint16_t* residual, uint16_t* y, float* u,
                                q4gsw_stream_t stream) {
  return guarded([&] {
    return adapters_fwd_impl(packed, N, K, group_size, false, plan, a, b, scale, L, r, x, M, bias, residual, y, u,
                             stream);
  });
}

q4gsw_status q4gsw_adapters_fwd_f32s(const void* packed, int N, int K, int group_size, const void* plan,
                                     const uint16_t* a, const uint16_t* b, const float* scale, int L, int r,
                                     const uint16_t* x, int M, const uint16_t* bias, const uint16_t* residual,
                                     uint16_t* y, float* u, q4gsw_stream_t stream) {
  return guarded([&] {
    return adapters_fwd_impl(packed, N, K, group_size, true, plan, a, b, scale, L, r, x, M, bias, residual, y, u,
                             stream);
  });
}

q4gsw_status q4gsw_adapters_bwd(const void* packed, int N, int K, int group_size, const void* plan, const uint16_t* a,
                                const uint16_t* b, const float* scale, int L, int r, const uint16_t* x,
                                const float* u, const uint16_t* d_y, int M, int accumulate, float* v, uint16_t* d_x,
                                float* d_a, float* d_b, q4gsw_stream_t stream) {
  return guarded([&] {
    return adapters_bwd_impl(packed, N, K, group_size, false, plan, a, b, scale, L, r, x, u, d_y, M, accumulate, v,
                             d_x, d_a, d_b, stream);
  });
}

q4gsw_status q4gsw_adapters_bwd_f32s(const void* packed, int N, int K, int group_size, const void* plan,
                                     const uint16_t* a, const uint16_t* b, const float* scale, int L, int r,
                                     const uint16_t* x, const float* u, const uint16_t* d_y, int M, int accumulate,
                                     float* v, uint16_t* d_x, float* d_a, float* d_b, q4gsw_stream_t stream) {
  return guarded([&] {
    return adapters_bwd_impl(packed, N, K, group_size, true, plan, a, b, scale, L, r, x, u, d_y, M, accumulate, v,
                             d_x, d_a, d_b, stream);
  });
}

q4gsw_status q4gsw_norms_fwd(const uint16_t* stream_in, const uint16_t* block, const uint16_t* w_post,
                             const uint16_t* gate, int gate_rows, float residual_scale, const uint16_t* w_pre,
                             float weight_offset, float eps, int M, int D, uint16_t* h_out, uint16_t* x,
                             q4gsw_stream_t stream) {
  return guarded([&]() -> q4gsw_status {
    const q4gsw_status st = check_norms(M, D, residual_scale, weight_offset, eps);
    if (st != Q4GSW_OK) return st;
    if (gate_rows != 0 && gate_rows != 1) return Q4GSW_ERR_UNSUPPORTED;
    if (M == 0) {
      set_route("empty");
      return Q4GSW_OK;
    }
    if (!stream_in || (!h_out && !x) || (!x) != (!w_pre) || (!block && (w_post || gate))) return Q4GSW_ERR_NULL;
    if (!aligned16(stream_in) || !aligned16(block) || !aligned16(w_post) || !aligned16(gate) || !aligned16(w_pre) ||
        !aligned16(h_out) || !aligned16(x))
      return Q4GSW_ERR_ALIGN;
    NormsArgs n = {};
    n.h = h(stream_in);
    n.block = h(block);
    n.w_post = h(w_post);
    n.gate = h(gate);
    n.w_pre = h(w_pre);
    n.h_out = h(h_out);
    n.x = h(x);
    n.residual_scale = residual_scale;
    n.weight_offset = weight_offset;
    n.eps = eps;
    n.gate_rows = gate_rows;
    n.M = M;
    n.D = D;
    char route[160] = "";
    const cudaError_t e = launch_norms_fwd(n, stream, route, sizeof(route));
    set_route(route);
    return from_cuda(e);
  });
}

size_t q4gsw_norms_workspace_bytes(int M, int D) {
  return check_norms(M, D, 1.f, 0.f, 0.f) == Q4GSW_OK ? norms_workspace_bytes(M, D) : 0;
}

q4gsw_status q4gsw_norms_bwd(const uint16_t* h_out, const uint16_t* d_x, const uint16_t* d_h, const uint16_t* block,
                             const uint16_t* w_post, const uint16_t* gate, int gate_rows, float residual_scale,
                             const uint16_t* w_pre, float weight_offset, float eps, int M, int D, uint16_t* d_residual,
                             uint16_t* d_block, uint16_t* d_gate_rows, float* d_w_pre, float* d_w_post, float* d_gate,
                             void* workspace, size_t workspace_bytes, q4gsw_stream_t stream) {
  return guarded([&]() -> q4gsw_status {
    const q4gsw_status st = check_norms(M, D, residual_scale, weight_offset, eps);
    if (st != Q4GSW_OK) return st;
    if (gate_rows != 0 && gate_rows != 1) return Q4GSW_ERR_UNSUPPORTED;
    if (!aligned16(d_w_pre) || !aligned16(d_w_post) || !aligned16(d_gate)) return Q4GSW_ERR_ALIGN;
    if (M == 0) {
      set_route("empty");
      for (float* p : {d_w_pre, d_w_post, d_gate}) {
        if (!p) continue;
        const cudaError_t e = cudaMemsetAsync(p, 0, sizeof(float) * (size_t)D, stream);
        if (e != cudaSuccess) return from_cuda(e);
      }
      return Q4GSW_OK;
    }
    const bool sums = d_w_pre || d_w_post || d_gate;
    const bool token_gate = gate && gate_rows;
    // what goes together: the pre norm's three, the block and what follows it
    if (!d_residual || (!d_x && !d_h) || (!d_x) != (!w_pre) || (d_x && !h_out)) return Q4GSW_ERR_NULL;
    if ((!block && (w_post || gate)) || (!block) != (!d_block) || token_gate != (d_gate_rows != nullptr))
      return Q4GSW_ERR_NULL;
    if ((d_w_pre && !w_pre) || (d_w_post && !w_post) || (d_gate && (!gate || gate_rows)) || (sums && !workspace))
      return Q4GSW_ERR_NULL;
    if (!aligned16(h_out) || !aligned16(d_x) || !aligned16(d_h) || !aligned16(block) || !aligned16(w_post) ||
        !aligned16(gate) || !aligned16(w_pre) || !aligned16(d_residual) || !aligned16(d_block) ||
        !aligned16(d_gate_rows) || !aligned16(workspace))
      return Q4GSW_ERR_ALIGN;
    if (sums && workspace_bytes < norms_workspace_bytes(M, D)) return Q4GSW_ERR_SIZE;
    NormsArgs n = {};
    n.h = h(h_out);
    n.block = h(block);
    n.w_post = h(w_post);
    n.gate = h(gate);
    n.w_pre = h(w_pre);
    n.d_x = h(d_x);
    n.d_h = h(d_h);
    n.h_out = h(d_residual);
    n.x = h(d_block);
    n.d_gate_rows = h(d_gate_rows);
    n.d_w_pre = d_w_pre;
    n.d_w_post = d_w_post;
    n.d_gate = d_gate;
    n.part = sums ? static_cast<float*>(workspace) : nullptr;
    n.residual_scale = residual_scale;
    n.weight_offset = weight_offset;
    n.eps = eps;
    n.gate_rows = gate_rows;
    n.M = M;
    n.D = D;
    char route[160] = "";
    const cudaError_t e = launch_norms_bwd(n, stream, route, sizeof(route));
    set_route(route);
    return from_cuda(e);
  });
}

size_t q4gsw_grad_table_bytes(int count, const int64_t* sizes) {
  return count < 1 || count > 65536 || !sizes ? 0 : grad_table_bytes(count, sizes);
}

q4gsw_status q4gsw_grad_table(int count, const void* const* grads, const int* half_grads, void* const* outs,
                              const int* half_outs, const int64_t* sizes, void* table, size_t table_bytes) {
  return guarded([&]() -> q4gsw_status {
    if (count < 1 || count > 65536) return Q4GSW_ERR_SHAPE;
    if (!grads || !half_grads || !sizes || !table || (!outs) != (!half_outs)) return Q4GSW_ERR_NULL;
    for (int i = 0; i < count; ++i) {
      if (sizes[i] < 0) return Q4GSW_ERR_SHAPE;
      if ((half_grads[i] != 0 && half_grads[i] != 1) || (outs && half_outs[i] != 0 && half_outs[i] != 1))
        return Q4GSW_ERR_UNSUPPORTED;
      if (sizes[i] == 0) continue;
      if (!grads[i] || (outs && !outs[i])) return Q4GSW_ERR_NULL;
      if ((reinterpret_cast<uintptr_t>(grads[i]) & (half_grads[i] ? 1u : 3u)) ||
          (outs && (reinterpret_cast<uintptr_t>(outs[i]) & (half_outs[i] ? 1u : 3u))))
        return Q4GSW_ERR_ALIGN;
    }
    const size_t need = grad_table_bytes(count, sizes);
    if (need == 0 || table_bytes < need) return Q4GSW_ERR_SIZE;
    grad_table_fill(count, grads, half_grads, outs, half_outs, sizes, table, need);
    return Q4GSW_OK;
  });
}

size_t q4gsw_grad_workspace_bytes(void) { return grad_workspace_bytes(); }

static q4gsw_status check_grad_call(const void* table, size_t table_bytes, float inv_scale, const float* norm,
                                    const void* workspace, size_t workspace_bytes) {
  if (!std::isfinite(inv_scale)) return Q4GSW_ERR_SHAPE;
  const bool few = table_bytes <= kGradRecordBytes * kGradFewRecords;
  if (!table || !norm || (!workspace && !few)) return Q4GSW_ERR_NULL;
  if (!aligned16(table) || !word(norm) || !aligned16(workspace)) return Q4GSW_ERR_ALIGN;
  if (table_bytes < kGradRecordBytes || table_bytes % kGradRecordBytes || table_bytes / kGradRecordBytes > 0x7fffffff ||
      (!few && workspace_bytes < grad_workspace_bytes()))
    return Q4GSW_ERR_SIZE;
  return Q4GSW_OK;
}

q4gsw_status q4gsw_grad_norm(const void* table, size_t table_bytes, float inv_scale, float* norm, void* workspace,
                             size_t workspace_bytes, q4gsw_stream_t stream) {
  return guarded([&] {
    const q4gsw_status st = check_grad_call(table, table_bytes, inv_scale, norm, workspace, workspace_bytes);
    if (st != Q4GSW_OK) return st;
    char route[160] = "";
    const cudaError_t e = launch_grad_norm(table, table_bytes, inv_scale, norm, workspace, stream, route, sizeof(route));
    set_route(route);
    return from_cuda(e);
  });
}

q4gsw_status q4gsw_grad_clip(const void* table, size_t table_bytes, float max_norm, float inv_scale, float* norm,
                             void* workspace, size_t workspace_bytes, q4gsw_stream_t stream) {
  return guarded([&] {
    if (!(max_norm > 0.f)) return Q4GSW_ERR_SHAPE;
    const q4gsw_status st = check_grad_call(table, table_bytes, inv_scale, norm, workspace, workspace_bytes);
    if (st != Q4GSW_OK) return st;
    char route[160] = "";
    const cudaError_t e = launch_grad_clip(table, table_bytes, max_norm, inv_scale, norm, workspace, stream, route, sizeof(route));
    set_route(route);
    return from_cuda(e);
  });
}

}  // extern "C"
