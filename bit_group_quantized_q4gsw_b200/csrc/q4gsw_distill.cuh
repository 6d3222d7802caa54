// q4gsw_distill.cuh - distillation from a teacher's top logits (sm_100a): the
// loss, the row's log-sum-exp and the gradient of the student's logits.
// Included once, by q4gsw_gemm_sm100.cu, which owns the device error word.
//
// Row m, temperature T, teacher entries (i_j, t_j), j < k:
//   q = softmax_j(t_j / T),  lse = log sum_i exp(z_i / T)
//   loss = T^2 sum_j q_j (log q_j - z[i_j] / T + lse)
//   d_z[i] = d_loss T (exp(z_i / T - lse) - sum of q_j with i_j = i)
//
// The rows are long (V tokens) and each logit is used for one exponential or
// two, so the kernels are streams: what they cost is the bytes of the logits
// and of the gradient.  A cluster of C CTAs shares a row.  Each thread issues
// the 16-byte loads of 32 logits at once, the CTA's (max, sum of exp) pairs are
// combined through shuffles and shared memory, and the C pairs of a row through
// distributed shared memory, in rank order.  Where a CTA's slice of the row
// fits its registers (V <= 8 x 8192), the gradient is computed from the
// registers that the sum was computed from: the logits cross the memory system
// once.  Longer rows are read a second time, shortly after the first, from L2.
//
// The gradient is first written as coef p for every token; the k teacher
// tokens are then written again as coef (p - q), in fp32 until the one
// rounding.  Every CTA does that for the tokens of its own slice, after a
// barrier, so the order of the two writes is fixed.
#pragma once

namespace q4gsw {
namespace distill {

constexpr int kThreads = 256;
constexpr int kPer = 32;                     // logits per thread and tile
constexpr int kTile = kThreads * kPer;       // 8192 logits
constexpr int kMaxK = 1024;                  // teacher entries per row
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Mode { kResident = 0, kStream = 1, kGradOnly = 2 };

__device__ __forceinline__ float ex2(float x) {   // 2^x, relative error 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (maximum, sum of 2^((x - maximum) c)) of a set of logits; an empty set (or
// one of -infinity alone) is (-infinity, 0).
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ MaxSum combine(MaxSum a, MaxSum b, float c) {
  const float m = fmaxf(a.m, b.m), r = finite_ref(m);
  return {m, a.s * ex2((a.m - r) * c) + b.s * ex2((b.m - r) * c)};
}

// One 16-byte vector of logits -> fp32 values.
template <bool HALF>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[HALF ? 8 : 4]) {
  if constexpr (HALF) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = __half22float2(u32_as_h2(w[j]));
      f[2 * j] = p.x;
      f[2 * j + 1] = p.y;
    }
  } else {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
}

template <bool HALF>
__device__ __forceinline__ float logit_at(const void* row, int i) {
  return HALF ? __half2float(static_cast<const __half*>(row)[i]) : static_cast<const float*>(row)[i];
}

// grid = M * C CTAs, cluster = (C, 1, 1) (kGradOnly: no cluster).  CTA `rank`
// of row m owns the 16-byte vectors [rank VV / C, (rank + 1) VV / C) of the row
// (VV = V / E; kGradOnly: one tile of kTile logits).
template <int MODE, bool HALF>
__global__ void __launch_bounds__(kThreads, 4) q4gsw_distill_kernel(const DistillArgs a, int C) {
  constexpr int E = HALF ? 8 : 4;         // logits per vector
  constexpr int NV = kPer / E;            // vectors per thread and tile
  __shared__ int s_idx[kMaxK];            // token id, -1: padding
  __shared__ float s_q[kMaxK];            // teacher logit, then q
  __shared__ MaxSum s_warp[kThreads / 32];
  __shared__ MaxSum s_cta;
  __shared__ float s_top, s_log_total;    // teacher: maximum; log of the sum of exponentials
  __shared__ int s_has;

  griddep_launch_dependents();
  const int m = blockIdx.x / C, rank = blockIdx.x % C;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int V = a.V, k = a.k;
  const float inv_t = 1.f / a.temperature, c = kLog2e / a.temperature;
  const int VV = V / E;
  const int v_begin = MODE == kGradOnly ? rank * (kTile / E) : (int)((long long)rank * VV / C);
  const int v_end = MODE == kGradOnly ? min(VV, v_begin + kTile / E) : (int)((long long)(rank + 1) * VV / C);
  const char* row = static_cast<const char*>(a.logits) + (size_t)m * V * (HALF ? 2 : 4);
  const uint4* rowv = reinterpret_cast<const uint4*>(row);
  const bool want_grad = MODE == kGradOnly || a.grad != nullptr;
  griddep_wait();

  // logits past the end of the slice: -infinity, which adds nothing
  const uint4 fill = HALF ? make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u)
                          : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  auto load_tile = [&](int base, uint4 (&x)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = base + i * kThreads + threadIdx.x;
      x[i] = at < v_end ? ldg_stream_v4(rowv + at) : fill;
    }
  };
  uint4 x[NV];
  if (MODE != kStream) load_tile(v_begin, x);

  // ---- teacher softmax (warp 0), while the logits are on their way
  if (warp == 0) {
    const int32_t* idx = a.indices + (size_t)m * k;
    const size_t t0 = (size_t)m * k;
    float top = -INFINITY;
    bool some = false, bad = false;
    for (int j = lane; j < k; j += 32) {
      int id = idx[j];
      float t = a.half_teacher ? __half2float(static_cast<const __half*>(a.teacher)[t0 + j])
                               : static_cast<const float*>(a.teacher)[t0 + j];
      if (id < 0 || id >= V) {
        bad |= id != -1;
        id = -1;
        t = -INFINITY;
      }
      s_idx[j] = id;
      s_q[j] = t;
      some |= t != -INFINITY;
      top = fmaxf(top, t);
    }
    some = __any_sync(0xffffffffu, some);
    if (__any_sync(0xffffffffu, bad) && lane == 0 && rank == 0) atomicOr(&g_device_error, kIndexErrorBit);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float total = 0.f;
    for (int j = lane; j < k; j += 32) total += ex2((s_q[j] - top) * c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) {
      s_has = some;
      s_top = top;
      s_log_total = logf(total);
    }
    // the teacher's logits stay for the loss (rank 0); q is ex2((t - top) c) / total
    s_cta.s = total;
    __syncwarp();
  }
  __syncthreads();
  const bool has = s_has != 0;
  const float top = s_top, inv_total = 1.f / s_cta.s;
  const float coef = want_grad ? a.d_loss[m] * a.temperature : 0.f;
  __syncthreads();   // s_cta is written again below

  // ---- (max, sum of exponentials) of the row
  float ref = 0.f, scale = 0.f;   // p_i = 2^((z_i - ref) c) scale
  if (MODE == kGradOnly) {
    ref = a.lse_in[m] * a.temperature;   // z_i / T - lse = (z_i - lse T) / T
    scale = 1.f;
  } else {
    MaxSum mine{-INFINITY, 0.f};
    auto add_tile = [&](const uint4 (&t)[NV]) {
      float top_t = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[E];
        unpack<HALF>(t[i], f);
#pragma unroll
        for (int e = 0; e < E; ++e) top_t = fmaxf(top_t, f[e]);
      }
      const float mx = fmaxf(mine.m, top_t), r = finite_ref(mx);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[E];
        unpack<HALF>(t[i], f);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          s0 += ex2((f[e] - r) * c);
          s1 += ex2((f[e + 1] - r) * c);
        }
      }
      mine = {mx, mine.s * ex2((mine.m - r) * c) + (s0 + s1)};
    };
    if (MODE == kResident) {
      add_tile(x);
    } else {
      for (int base = v_begin; base < v_end; base += kTile / E) {
        load_tile(base, x);
        add_tile(x);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      mine = combine(mine, {__shfl_xor_sync(0xffffffffu, mine.m, o), __shfl_xor_sync(0xffffffffu, mine.s, o)}, c);
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
      MaxSum t = s_warp[0];
      for (int w = 1; w < kThreads / 32; ++w) t = combine(t, s_warp[w], c);
      s_cta = t;
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (C > 1) cluster.sync();
    else __syncthreads();
    MaxSum all{-INFINITY, 0.f};
    for (int q = 0; q < C; ++q) all = combine(all, C > 1 ? *cluster.map_shared_rank(&s_cta, q) : s_cta, c);
    if (C > 1) cluster.sync();   // no CTA leaves while another reads its pair
    ref = all.m;
    scale = 1.f / all.s;
    if (rank == 0 && warp == 0) {
      // (all.m - all.m) is 0, or NaN where the row's maximum is not finite
      const float lse = fmaf(all.m, inv_t, logf(all.s)) + (all.m - all.m);
      float part = 0.f;
      if (has) {
        for (int j = lane; j < k; j += 32) {
          const float lt = (s_q[j] - top) * inv_t - s_log_total;   // log q_j
          const float q = ex2((s_q[j] - top) * c) * inv_total;
          // a weight of zero adds nothing, whatever its token's logit (a NaN
          // weight, from a NaN of the teacher, is added)
          if (s_idx[j] >= 0 && !(q == 0.f)) part += q * (lt - logit_at<HALF>(row, s_idx[j]) * inv_t + lse);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if (lane == 0) {
        a.lse[m] = lse;
        a.loss[m] = part * a.temperature * a.temperature;
      }
    }
  }
  if (!want_grad) return;

  // ---- gradient: coef p for every token of the slice, then the teacher's tokens again
  __half* grow = a.grad + (size_t)m * V;
  auto store_tile = [&](int base, const uint4 (&t)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = base + i * kThreads + threadIdx.x;
      if (at >= v_end) continue;
      float f[E];
      unpack<HALF>(t[i], f);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = has ? coef * (ex2((f[e] - ref) * c) * scale) : 0.f;
      if constexpr (HALF) {
        *reinterpret_cast<uint4*>(grow + (size_t)at * 8) =
            make_uint4(h2_as_u32(__floats2half2_rn(f[0], f[1])), h2_as_u32(__floats2half2_rn(f[2], f[3])),
                       h2_as_u32(__floats2half2_rn(f[4], f[5])), h2_as_u32(__floats2half2_rn(f[6], f[7])));
      } else {
        *reinterpret_cast<uint2*>(grow + (size_t)at * 4) =
            make_uint2(h2_as_u32(__floats2half2_rn(f[0], f[1])), h2_as_u32(__floats2half2_rn(f[2], f[3])));
      }
    }
  };
  if (MODE != kStream) {
    store_tile(v_begin, x);
  } else {
    for (int base = v_begin; base < v_end; base += kTile / E) {
      load_tile(base, x);
      store_tile(base, x);
    }
  }
  __syncthreads();
  if (!has) return;
  for (int j = threadIdx.x; j < k; j += kThreads) {
    const int id = s_idx[j];
    if (id < v_begin * E || id >= v_end * E) continue;   // padding, or another CTA's token
    float t = 0.f;   // every entry of this token, in the order of the list: each writes the same value
    for (int i = 0; i < k; ++i)
      if (s_idx[i] == id) t += ex2((s_q[i] - top) * c);
    const float p = ex2((logit_at<HALF>(row, id) - ref) * c) * scale;
    grow[id] = __float2half_rn(coef * (p - t * inv_total));
  }
}

}  // namespace distill

template <int MODE, bool HALF>
static cudaError_t distill_launch(const DistillArgs& a, int C, bool cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.M * (unsigned)C, 1, 1);
  cfg.blockDim = dim3(distill::kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, distill::q4gsw_distill_kernel<MODE, HALF>, a, C);
}

cudaError_t launch_distill_rows(const DistillArgs& a, bool half_logits, cudaStream_t stream, char* route,
                                int route_len) {
  using namespace distill;
  // CTAs per row: as many tiles as the row has (at most a cluster of 8), and
  // more, down to a quarter of a tile each, while the launch would leave SMs
  // without work.
  int C = 1;
  while (C < kMaxCluster && (long long)C * kTile < a.V) C *= 2;
  const bool resident = (long long)C * kTile >= a.V;
  const int sms = sm_count(current_device());
  while (C < kMaxCluster && (long long)a.M * C < 2LL * sms && a.V / (2 * C) >= kTile / 4) C *= 2;
  if (route)
    snprintf(route, route_len, "distill_%s launches=1 cluster=%d %s", a.grad ? "step" : "fwd", C,
             resident ? "resident" : "streamed");
  if (resident)
    return half_logits ? distill_launch<kResident, true>(a, C, true, stream)
                       : distill_launch<kResident, false>(a, C, true, stream);
  return half_logits ? distill_launch<kStream, true>(a, C, true, stream)
                     : distill_launch<kStream, false>(a, C, true, stream);
}

cudaError_t launch_distill_bwd(const DistillArgs& a, bool half_logits, cudaStream_t stream, char* route,
                               int route_len) {
  const int C = (a.V + distill::kTile - 1) / distill::kTile;
  if (route) snprintf(route, route_len, "distill_bwd launches=1 tiles=%d", C);
  return half_logits ? distill_launch<distill::kGradOnly, true>(a, C, false, stream)
                     : distill_launch<distill::kGradOnly, false>(a, C, false, stream);
}

}  // namespace q4gsw
