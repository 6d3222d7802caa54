// q4gsw_epilogue.cuh - what a product does with its finished fp32 sums: the
// output descriptors of the GEMV and GEMM kernels and the activations.
//
// Every product kernel is a template over its output descriptor:
//   OutSplit  fp32 rows, split over up to three buffers (the plain forward,
//             the fused Q/K/V projection, the input gradient);
//   Epi       fp16 rows, with the epilogue of a projection or of the gated
//             feed-forward block applied to the fp32 sums in registers;
//   EpiLow    fp16 rows of a projection with an adapter for every token
//             (q4gsw_lowrank.cuh).
// The epilogue adds no pass over memory: a projection followed by separate
// bias, activation and residual passes writes and re-reads its fp32 result
// (8 bytes an element) per pass; here each element is written once, in 2 bytes.
// With it and the plain fp32 product (us, replayed back to back on the same buffers
// at 1965 MHz): a token of 2048 x 8192 with residual 6.7 and 6.6; with bias and
// residual 16 tokens of 14336 x 4096 13.8 and 13.7, 508 tokens of 2048 x 8192 19.8
// and 19.5, 512 tokens of 16384 x 2048 30.0 and 33.6 (28.6 without either); gated
// there 30.4.
//
// The gated block's weight interleaves its two matrices row by row (feature
// 2 j = gate row j, 2 j + 1 = up row j; the packed layout already stores such
// a pair of rows in one byte row), so the two sums a gated output needs are
// neighbours in every kernel's output tile and no kernel exchanges anything.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "q4gsw_common.cuh"
#include "q4gsw_internal.h"

namespace q4gsw {

// 1 / (1 + e^-z).  The fast exponential is within 2 + 1.2 |z| units in the last
// place (at most 2^-23 of its value each) and the quotient within 2: 2^-19 at |z| =
// 10, 2^-16 at the far end of the negative side, still far below the fp16 rounding of
// every result that uses it.
// Past a denominator of 2^126 (z < -87) the quotient is 0, its limit.
__device__ __forceinline__ float sigmoid_f32(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// A saved value that passed the fp16 range is an infinity; products of it with
// the zeros that the activations reach there would be NaN.  2^42 stands for it:
// act and act' have reached their limits, z^3 is in the fp32 range, and what is
// multiplied by it rounds to an fp16 infinity from the least fp16 step on.  A NaN
// stays, and finite fp16 values are not touched.
__device__ __forceinline__ float within(float z) {
  float v;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(v) : "f"(z), "f"(4398046511104.f));   // min of |z|, z's sign
  return v;
}

// act(z) and, in `slope`, act'(z).
//   silu       z s,  s = 1 / (1 + e^-z);           s (1 + z (1 - s))
//   gelu_tanh  z s,  s = 1 / (1 + e^-2v) = (1 + tanh v) / 2,
//              v = sqrt(2/pi) (z + 0.044715 z^3);  s + z s (1 - s) 2 v'
__device__ __forceinline__ float act_value(float z, int act) {
  if (act == kActNone) return z;
  if (act == kActSilu) return z * sigmoid_f32(z);
  const float v = 0.7978845608028654f * fmaf(0.044715f * z * z, z, z);
  return z * sigmoid_f32(2.f * v);
}
// (of a finite z: `within` for saved values)
__device__ __forceinline__ float act_value_slope(float z, int act, float& slope) {
  if (act == kActNone) {
    slope = 1.f;
    return z;
  }
  if (act == kActSilu) {
    const float s = sigmoid_f32(z);
    slope = s * fmaf(z, 1.f - s, 1.f);
    return z * s;
  }
  const float z2 = z * z;
  const float s = sigmoid_f32(1.5957691216057308f * fmaf(0.044715f * z2, z, z));
  slope = fmaf(z * s * (1.f - s), 1.5957691216057308f * fmaf(0.134145f, z2, 1.f), s);
  return z * s;
}

// Whether a product reads its activations before it waits for the kernel in front.
template <typename Out>
constexpr bool kReadsEarly = std::is_same_v<Out, EpiLow>;
// Whether its outputs are fp16.
template <typename Out>
constexpr bool kHalfOut = std::is_same_v<Out, Epi> || std::is_same_v<Out, EpiLow>;

// ---------------------------------------------------------------- OutSplit
// What an epilogue reads before it stores: nothing here.
struct NoOperand {};
__device__ __forceinline__ NoOperand epi_load4(const OutSplit&, size_t, int) { return {}; }

// four consecutive features n .. n + 3 (n % 4 == 0) of token m
__device__ __forceinline__ void epi_store4(const OutSplit& o, size_t m, int n, float4 v, NoOperand) {
  float* dst;
  if (n < o.n1) dst = o.y0 + m * o.n1 + n;
  else if (n < o.n2) dst = o.y1 + m * (o.n2 - o.n1) + (n - o.n1);
  else dst = o.y2 + m * (o.N - o.n2) + (n - o.n2);
  *reinterpret_cast<float4*>(dst) = v;
}

// ---------------------------------------------------------------- Epi
// Bias and residual of four features, loaded ahead of the sums they are added
// to.  The residual may be the output buffer itself (each element is read and
// then written by one thread), so it is not read through the non-coherent path.
struct EpiOperand {
  uint2 bias, res;
};
__device__ __forceinline__ EpiOperand epi_load4(const Epi& o, size_t m, int n) {
  EpiOperand q{make_uint2(0u, 0u), make_uint2(0u, 0u)};
  if (o.bias) q.bias = *reinterpret_cast<const uint2*>(o.bias + n);
  if (o.res) q.res = *reinterpret_cast<const uint2*>(o.res + m * o.N + n);
  return q;
}

__device__ __forceinline__ float4 half4_f32(uint2 v) {
  const float2 a = __half22float2(u32_as_h2(v.x)), b = __half22float2(u32_as_h2(v.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint2 f32_half4(float4 v) {
  return make_uint2(h2_as_u32(__floats2half2_rn(v.x, v.y)), h2_as_u32(__floats2half2_rn(v.z, v.w)));
}

__device__ __forceinline__ void epi_store4(const Epi& o, size_t m, int n, float4 v, const EpiOperand& q) {
  if (o.gated) {
    // (g, u) pairs of gated features n / 2 and n / 2 + 1
    if (o.z) *reinterpret_cast<uint2*>(o.z + m * o.N + n) = f32_half4(v);
    const __half2 h = __floats2half2_rn(act_value(v.x, o.act) * v.y, act_value(v.z, o.act) * v.w);
    *reinterpret_cast<uint32_t*>(o.y + m * (o.N >> 1) + (n >> 1)) = h2_as_u32(h);
    return;
  }
  const float4 b = half4_f32(q.bias), r = half4_f32(q.res);
  v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
  if (o.z) *reinterpret_cast<uint2*>(o.z + m * o.N + n) = f32_half4(v);
  v = make_float4(act_value(v.x, o.act) + r.x, act_value(v.y, o.act) + r.y, act_value(v.z, o.act) + r.z,
                  act_value(v.w, o.act) + r.w);
  *reinterpret_cast<uint2*>(o.y + m * o.N + n) = f32_half4(v);
}

// two consecutive features n, n + 1 (n even): the GEMV kernels' store
__device__ __forceinline__ void epi_store2(const Epi& o, size_t m, int n, float v0, float v1) {
  const size_t at = m * o.N + n;
  if (o.gated) {
    if (o.z) *reinterpret_cast<uint32_t*>(o.z + at) = h2_as_u32(__floats2half2_rn(v0, v1));
    o.y[m * (o.N >> 1) + (n >> 1)] = __float2half_rn(act_value(v0, o.act) * v1);
    return;
  }
  if (o.bias) {
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(o.bias + n));
    v0 += b.x;
    v1 += b.y;
  }
  if (o.z) *reinterpret_cast<uint32_t*>(o.z + at) = h2_as_u32(__floats2half2_rn(v0, v1));
  v0 = act_value(v0, o.act);
  v1 = act_value(v1, o.act);
  if (o.res) {
    const float2 r = __half22float2(*reinterpret_cast<const __half2*>(o.res + at));
    v0 += r.x;
    v1 += r.y;
  }
  *reinterpret_cast<uint32_t*>(o.y + at) = h2_as_u32(__floats2half2_rn(v0, v1));
}

// ---------------------------------------------------------------- EpiLow
// (the term is in the sums by then)
__device__ __forceinline__ EpiOperand epi_load4(const EpiLow& o, size_t m, int n) {
  EpiOperand q{make_uint2(0u, 0u), make_uint2(0u, 0u)};
  if (o.bias) q.bias = *reinterpret_cast<const uint2*>(o.bias + n);
  if (o.res) q.res = *reinterpret_cast<const uint2*>(o.res + m * o.N + n);
  return q;
}
__device__ __forceinline__ void epi_store4(const EpiLow& o, size_t m, int n, float4 v, const EpiOperand& q) {
  const float4 b = half4_f32(q.bias), r = half4_f32(q.res);
  *reinterpret_cast<uint2*>(o.y + m * o.N + n) =
      f32_half4(make_float4(v.x + b.x + r.x, v.y + b.y + r.y, v.z + b.z + r.z, v.w + b.w + r.w));
}

}  // namespace q4gsw
