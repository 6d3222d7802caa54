// q4gsw_layer_api.cu - the extern "C" entry points declared in
// include/q4gsw_layer.h: argument checks, route strings and launches.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>

#include "../../include/q4gsw_layer.h"
#include "q4gsw_api_common.h"
#include "q4gsw_common.cuh"
#include "q4gsw_internal.h"

using namespace q4gsw;

namespace {

// No C++ exception may cross the C boundary (a launcher's first-use cache can
// throw std::system_error).
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

q4gsw_status check_gated_shape(int F, int K, int gs) {
  if (F <= 0 || F > 0x3fffffff || F % 4) return Q4GSW_ERR_SHAPE;
  if (F % 8) return Q4GSW_ERR_ALIGN;   // 16-byte rows of h
  return check_weight_shape(2 * F, K, gs);
}

bool gated_act(int act) { return act == Q4GSW_ACT_SILU || act == Q4GSW_ACT_GELU_TANH; }
bool any_act(int act) { return act == Q4GSW_ACT_NONE || gated_act(act); }

q4gsw_status prepack_gated_impl(const uint8_t* codes_gate, const void* scales_gate, const uint8_t* codes_up,
                                const void* scales_up, int F, int K, int gs, bool f32s, void* packed,
                                size_t packed_bytes, q4gsw_stream_t stream) {
  if (!codes_gate || !scales_gate || !codes_up || !scales_up || !packed) return Q4GSW_ERR_NULL;
  const q4gsw_status st = check_gated_shape(F, K, gs);
  if (st != Q4GSW_OK) return st;
  if (!aligned16(codes_gate) || !aligned16(scales_gate) || !aligned16(codes_up) || !aligned16(scales_up) ||
      !aligned16(packed))
    return Q4GSW_ERR_ALIGN;
  if (packed_bytes < layout_of(2 * F, K, gs, f32s ? 4 : 2).total_bytes) return Q4GSW_ERR_SIZE;
  uint32_t flag = 0;
  set_route(f32s ? "prepack_gated_f32s" : "prepack_gated");
  const q4gsw_status e = from_cuda(launch_prepack_gated(codes_gate, scales_gate, codes_up, scales_up, F, K, gs, f32s,
                                                        packed, stream, &flag));
  if (e != Q4GSW_OK) return e;
  return flag ? Q4GSW_ERR_CODE_RANGE : Q4GSW_OK;
}

q4gsw_status gated_fwd_impl(const void* packed, int F, int K, int gs, bool f32s, const uint16_t* x, int M, int act,
                            uint16_t* y, uint16_t* gu, q4gsw_stream_t stream) {
  if (M < 0) return Q4GSW_ERR_SHAPE;
  const q4gsw_status st = check_gated_shape(F, K, gs);
  if (st != Q4GSW_OK) return st;
  if (!gated_act(act)) return Q4GSW_ERR_UNSUPPORTED;
  if (M == 0) {
    set_route("empty");
    return Q4GSW_OK;
  }
  if (!packed || !x || !y) return Q4GSW_ERR_NULL;
  if (!aligned16(packed) || !aligned16(x) || !aligned16(y) || !aligned16(gu)) return Q4GSW_ERR_ALIGN;
  const Epi out{h(y), h(gu), nullptr, nullptr, 2 * F, act, 1};
  char inner[128] = "", route[160];
  const cudaError_t e = launch_product_epi(false, packed, 2 * F, K, gs, f32s, x, M, out, stream, inner, sizeof(inner));
  snprintf(route, sizeof(route), "gated %s", inner);
  set_route(route);
  return from_cuda(e);
}

q4gsw_status gated_bwd_impl(const void* packed, int F, int K, int gs, bool f32s, const uint16_t* gu,
                            const uint16_t* d_h, int M, int act, uint16_t* d_gu, uint16_t* d_x,
                            q4gsw_stream_t stream) {
  if (M < 0) return Q4GSW_ERR_SHAPE;
  const q4gsw_status st = check_gated_shape(F, K, gs);
  if (st != Q4GSW_OK) return st;
  if (!gated_act(act)) return Q4GSW_ERR_UNSUPPORTED;
  if (M == 0) {
    set_route("empty");
    return Q4GSW_OK;
  }
  if (!packed || !gu || !d_h || !d_gu || !d_x) return Q4GSW_ERR_NULL;
  if (!aligned16(packed) || !aligned16(gu) || !aligned16(d_h) || !aligned16(d_gu) || !aligned16(d_x))
    return Q4GSW_ERR_ALIGN;
  cudaError_t e = launch_gated_grad(h(gu), h(d_h), M, F, act, h(d_gu), stream);
  if (e != cudaSuccess) return from_cuda(e);
  const Epi out{h(d_x), nullptr, nullptr, nullptr, K, kActNone, 0};
  char inner[128] = "", route[160];
  e = launch_product_epi(true, packed, 2 * F, K, gs, f32s, d_gu, M, out, stream, inner, sizeof(inner));
  snprintf(route, sizeof(route), "gated grad launches=1 + %s", inner);   // every part counts its own
  set_route(route);
  return from_cuda(e);
}

q4gsw_status act_fwd_impl(const void* packed, int N, int K, int gs, bool f32s, const uint16_t* x, int M,
                          const uint16_t* bias, int act, const uint16_t* residual, uint16_t* y, uint16_t* z,
                          q4gsw_stream_t stream) {
  if (M < 0) return Q4GSW_ERR_SHAPE;
  const q4gsw_status st = check_weight_shape(N, K, gs);
  if (st != Q4GSW_OK) return st;
  if (!any_act(act)) return Q4GSW_ERR_UNSUPPORTED;
  if (M == 0) {
    set_route("empty");
    return Q4GSW_OK;
  }
  if (!packed || !x || !y) return Q4GSW_ERR_NULL;
  if (!aligned16(packed) || !aligned16(x) || !aligned16(bias) || !aligned16(residual) || !aligned16(y) ||
      !aligned16(z))
    return Q4GSW_ERR_ALIGN;
  const Epi out{h(y), h(z), h(bias), h(residual), N, act, 0};
  char inner[128] = "", route[160];
  const cudaError_t e = launch_product_epi(false, packed, N, K, gs, f32s, x, M, out, stream, inner, sizeof(inner));
  snprintf(route, sizeof(route), "linear_act %s", inner);
  set_route(route);
  return from_cuda(e);
}

q4gsw_status act_bwd_impl(const void* packed, int N, int K, int gs, bool f32s, const uint16_t* z,
                          const uint16_t* d_y, int M, int act, uint16_t* d_z, uint16_t* d_x, float* d_bias,
                          q4gsw_stream_t stream) {
  if (M < 0) return Q4GSW_ERR_SHAPE;
  const q4gsw_status st = check_weight_shape(N, K, gs);
  if (st != Q4GSW_OK) return st;
  if (!any_act(act)) return Q4GSW_ERR_UNSUPPORTED;
  if (!aligned16(d_bias)) return Q4GSW_ERR_ALIGN;
  if (M == 0) {
    set_route("empty");
    return d_bias ? from_cuda(cudaMemsetAsync(d_bias, 0, sizeof(float) * (size_t)N, stream)) : Q4GSW_OK;
  }
  const bool has_act = act != Q4GSW_ACT_NONE;
  if (!packed || !d_y || !d_x || (has_act && (!z || !d_z))) return Q4GSW_ERR_NULL;
  if (!aligned16(packed) || !aligned16(d_y) || !aligned16(d_x) || (has_act && (!aligned16(z) || !aligned16(d_z))))
    return Q4GSW_ERR_ALIGN;
  const bool grad = has_act || d_bias;
  if (grad) {
    const cudaError_t e = launch_act_grad(has_act ? h(z) : nullptr, h(d_y), M, N, act, has_act ? h(d_z) : nullptr,
                                          d_bias, stream);
    if (e != cudaSuccess) return from_cuda(e);
  }
  const Epi out{h(d_x), nullptr, nullptr, nullptr, K, kActNone, 0};
  char inner[128] = "", route[160];
  const cudaError_t e = launch_product_epi(true, packed, N, K, gs, f32s, has_act ? d_z : d_y, M, out, stream, inner,
                                           sizeof(inner));
  snprintf(route, sizeof(route), "linear_act %s%s", grad ? "grad launches=1 + " : "", inner);
  set_route(route);
  return from_cuda(e);
}

enum DistillCall { kFwd, kBwd, kStep };

q4gsw_status distill_impl(DistillCall call, DistillArgs a, int half_logits, q4gsw_stream_t stream) {
  if (a.M < 0 || a.V <= 0 || a.k < 1 || a.k > 1024) return Q4GSW_ERR_SHAPE;
  if (a.V % 4) return Q4GSW_ERR_SHAPE;
  if (a.V % 8) return Q4GSW_ERR_ALIGN;   // 16-byte vectors of logits and of the gradient
  // T^2 and 1 / T are factors: both within the normal fp32 range (NaN fails, too)
  if (!(a.temperature > 1e-18f && a.temperature < 1e18f)) return Q4GSW_ERR_SHAPE;
  // one item per row and tile of 8192 logits must count in 32 bits (the grids are no
  // larger than what is resident, up to 16 CTAs a row)
  const long long per_row = a.V / 8192 + 1 > 8 ? a.V / 8192 + 1 : 8;
  if (a.M > 0x7fffffffLL / per_row) return Q4GSW_ERR_SHAPE;
  if ((half_logits != 0 && half_logits != 1) || (a.half_teacher != 0 && a.half_teacher != 1))
    return Q4GSW_ERR_UNSUPPORTED;
  if (a.M == 0) {
    set_route("empty");
    return Q4GSW_OK;
  }
  if (!a.logits || !a.indices || !a.teacher) return Q4GSW_ERR_NULL;
  if (call == kBwd ? !a.lse_in : (!a.loss || !a.lse)) return Q4GSW_ERR_NULL;
  if (call != kFwd && (!a.d_loss || !a.grad)) return Q4GSW_ERR_NULL;
  auto word = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
  if (!aligned16(a.logits) || !aligned16(a.grad) || !word(a.indices) || !word(a.loss) || !word(a.lse) ||
      !word(a.lse_in) || !word(a.d_loss) || (reinterpret_cast<uintptr_t>(a.teacher) & (a.half_teacher ? 1u : 3u)))
    return Q4GSW_ERR_ALIGN;
  char route[160] = "";
  const cudaError_t e = call == kBwd ? launch_distill_bwd(a, half_logits != 0, stream, route, sizeof(route))
                                     : launch_distill_rows(a, half_logits != 0, stream, route, sizeof(route));
  set_route(route);
  return from_cuda(e);
}

}  // namespace

extern "C" {

q4gsw_status q4gsw_prepack_gated(const uint8_t* codes_gate, const uint16_t* scales_gate, const uint8_t* codes_up,
                                 const uint16_t* scales_up, int F, int K, int group_size, void* packed,
                                 size_t packed_bytes, q4gsw_stream_t stream) {
  return guarded([&] {
    return prepack_gated_impl(codes_gate, scales_gate, codes_up, scales_up, F, K, group_size, false, packed,
                              packed_bytes, stream);
  });
}

q4gsw_status q4gsw_prepack_gated_f32s(const uint8_t* codes_gate, const float* scales_gate, const uint8_t* codes_up,
                                      const float* scales_up, int F, int K, int group_size, void* packed,
                                      size_t packed_bytes, q4gsw_stream_t stream) {
  return guarded([&] {
    return prepack_gated_impl(codes_gate, scales_gate, codes_up, scales_up, F, K, group_size, true, packed,
                              packed_bytes, stream);
  });
}

q4gsw_status q4gsw_gated_fwd(const void* packed, int F, int K, int group_size, const uint16_t* x, int M, int act,
                             uint16_t* y, uint16_t* gu, q4gsw_stream_t stream) {
  return guarded([&] { return gated_fwd_impl(packed, F, K, group_size, false, x, M, act, y, gu, stream); });
}

q4gsw_status q4gsw_gated_fwd_f32s(const void* packed, int F, int K, int group_size, const uint16_t* x, int M, int act,
                                  uint16_t* y, uint16_t* gu, q4gsw_stream_t stream) {
  return guarded([&] { return gated_fwd_impl(packed, F, K, group_size, true, x, M, act, y, gu, stream); });
}

q4gsw_status q4gsw_gated_bwd(const void* packed, int F, int K, int group_size, const uint16_t* gu,
                             const uint16_t* d_h, int M, int act, uint16_t* d_gu, uint16_t* d_x,
                             q4gsw_stream_t stream) {
  return guarded([&] { return gated_bwd_impl(packed, F, K, group_size, false, gu, d_h, M, act, d_gu, d_x, stream); });
}

q4gsw_status q4gsw_gated_bwd_f32s(const void* packed, int F, int K, int group_size, const uint16_t* gu,
                                  const uint16_t* d_h, int M, int act, uint16_t* d_gu, uint16_t* d_x,
                                  q4gsw_stream_t stream) {
  return guarded([&] { return gated_bwd_impl(packed, F, K, group_size, true, gu, d_h, M, act, d_gu, d_x, stream); });
}

q4gsw_status q4gsw_linear_act_fwd(const void* packed, int N, int K, int group_size, const uint16_t* x, int M,
                                  const uint16_t* bias, int act, const uint16_t* residual, uint16_t* y, uint16_t* z,
                                  q4gsw_stream_t stream) {
  return guarded([&] {
    return act_fwd_impl(packed, N, K, group_size, false, x, M, bias, act, residual, y, z, stream);
  });
}

q4gsw_status q4gsw_linear_act_fwd_f32s(const void* packed, int N, int K, int group_size, const uint16_t* x, int M,
                                       const uint16_t* bias, int act, const uint16_t* residual, uint16_t* y,
                                       uint16_t* z, q4gsw_stream_t stream) {
  return guarded([&] {
    return act_fwd_impl(packed, N, K, group_size, true, x, M, bias, act, residual, y, z, stream);
  });
}

q4gsw_status q4gsw_linear_act_bwd(const void* packed, int N, int K, int group_size, const uint16_t* z,
                                  const uint16_t* d_y, int M, int act, uint16_t* d_z, uint16_t* d_x, float* d_bias,
                                  q4gsw_stream_t stream) {
  return guarded([&] {
    return act_bwd_impl(packed, N, K, group_size, false, z, d_y, M, act, d_z, d_x, d_bias, stream);
  });
}

q4gsw_status q4gsw_linear_act_bwd_f32s(const void* packed, int N, int K, int group_size, const uint16_t* z,
                                       const uint16_t* d_y, int M, int act, uint16_t* d_z, uint16_t* d_x,
                                       float* d_bias, q4gsw_stream_t stream) {
  return guarded([&] {
    return act_bwd_impl(packed, N, K, group_size, true, z, d_y, M, act, d_z, d_x, d_bias, stream);
  });
}

q4gsw_status q4gsw_distill_fwd(const void* logits, int half_logits, int M, int V, const int32_t* indices,
                               const void* teacher, int half_teacher, int k, float temperature, float* loss,
                               float* lse, q4gsw_stream_t stream) {
  return guarded([&] {
    return distill_impl(kFwd,
                        DistillArgs{logits, indices, teacher, nullptr, nullptr, loss, lse, nullptr, M, V, k,
                                    half_teacher, temperature, 1.f / temperature},
                        half_logits, stream);
  });
}

q4gsw_status q4gsw_distill_bwd(const void* logits, int half_logits, int M, int V, const float* lse,
                               const int32_t* indices, const void* teacher, int half_teacher, int k,
                               float temperature, const float* d_loss, uint16_t* d_logits, q4gsw_stream_t stream) {
  return guarded([&] {
    return distill_impl(kBwd,
                        DistillArgs{logits, indices, teacher, d_loss, lse, nullptr, nullptr, h(d_logits), M, V, k,
                                    half_teacher, temperature, 1.f / temperature},
                        half_logits, stream);
  });
}

q4gsw_status q4gsw_distill_step(const void* logits, int half_logits, int M, int V, const int32_t* indices,
                                const void* teacher, int half_teacher, int k, float temperature, const float* d_loss,
                                float* loss, float* lse, uint16_t* d_logits, q4gsw_stream_t stream) {
  return guarded([&] {
    return distill_impl(kStep,
                        DistillArgs{logits, indices, teacher, d_loss, nullptr, loss, lse, h(d_logits), M, V, k,
                                    half_teacher, temperature, 1.f / temperature},
                        half_logits, stream);
  });
}

}  // extern "C"
