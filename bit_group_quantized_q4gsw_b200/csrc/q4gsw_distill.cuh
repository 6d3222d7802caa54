// q4gsw_distill.cuh - distillation from a teacher's top logits (sm_100a): the
// loss, the row's log-sum-exp and the gradient of the student's logits.
// Included once, by q4gsw_gemm_sm100.cu, which owns the device error word.
//
// Row m, temperature T, teacher entries (i_j, t_j), j < k:
//   q = softmax_j(t_j / T),  lse = log sum_i exp(z_i / T)
//   loss = T^2 sum_j q_j (log q_j - z[i_j] / T + lse)
//   d_z[i] = d_loss T (exp(z_i / T - lse) - sum of q_j with i_j = i)
//
// The rows are long (V tokens) and each logit is used for one exponential: streams,
// whose floor is the bytes of the logits and of the gradient.  The gradient alone is
// near it (45.6 us, floor 40.2, for 2048 x 32000 in fp16); the step is bound by each
// row's chain of maximum, sum, exchange and gradient and by what it issues per logit
// (23.5 us, floor 15.0, for 512 x 32000), the loss of a few long rows by launch and
// latency (10.5 us, floor 5.9, for 37 x 262144).  So as many bytes as possible are
// kept in flight and as little as possible is issued per logit:
//  - a CTA of 128 threads keeps 64 logits of its part of a row in each thread's
//    registers, and from the sum on their weights in their place, from which the
//    gradient is a factor away: the logits cross the memory system once and each
//    costs one exponential (with a second one for the gradient 27.3 us instead
//    of 25.2 for the step of 512 x 32000); a cluster of up to eight CTAs holds a row
//    of 65536 tokens (longer rows take two launches and are read by both).  At 96
//    registers, five CTAs an SM, the step spills 48 bytes a thread, the fp32 loss 12;
//  - the launch holds as many CTAs as fit the SMs (five each) and each walks its
//    rows.  While a row is reduced and its gradient written, the next row's
//    logits, teacher entries and scalars are already on their way (cp.async
//    into shared memory, and registers that nothing touches before the next
//    row);
//  - the (max, sum of exp) pairs of a row's CTAs are exchanged by asynchronous
//    stores into each other's shared memory that count on a barrier there (a
//    cluster barrier would first wait for the gradient's stores), and added in
//    a fixed order; the buffers alternate between two rows, so nothing waits to
//    free them;
//  - the teacher's softmax is spread over the threads, one entry each, while the
//    row's logits arrive (in one warp, for all entries, it held up the row: 64
//    entries 54 us instead of 45 for the gradient of 2048 x 32000).
// The gradient is first written as coef p for every token; the k teacher
// tokens are then written again as coef (p - q), in fp32 until the one
// rounding.  Every CTA does that for the tokens of its own slice, after a
// barrier, so the order of the two writes is fixed.
#pragma once

namespace q4gsw {
namespace distill {

constexpr int kMaxCluster = 16;             // past 8: allowed by an attribute of the kernel
constexpr int kHoldCluster = 8;             // CTAs that hold a row between its loss and its gradient
constexpr int kThreads = 128, kWarps = 4;
constexpr int kPer = 64;                     // logits per thread and tile
constexpr int kTile = kThreads * kPer;       // 8192 logits
constexpr int kPerSm = 5;                    // resident CTAs per SM

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kHuge = 1e37f;   // |m c| beyond this: exponents from (x - m) c, which does not overflow to NaN

__device__ __forceinline__ float ex2(float x) {   // 2^x, relative error 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (maximum m, sum of the weights of x against m) of a set of logits; an empty
// set (or one of -infinity alone) is (-infinity, 0).
struct alignas(8) MaxSum {
  float m, s;
};
// Weight of x against a maximum m: 2^(x c - base), base = m c rounded.  The
// exponent is one fused multiply-add, exact but for its own rounding, and what
// rounding m c changed is the same factor for all of a row.  Where m c is near
// the end of the fp32 range (a row masked with the type's lowest value) it is
// (x - m) c; an m of -infinity stands for a base of 0.
// The product is rounded by name wherever a base is formed or left: written as
// an operator it may be contracted into the subtraction behind it, and the sum
// then moves by 2^(m c - base), another factor for every warp's and CTA's
// maximum (2.9e-3 of p at logits around 2e4, T = 0.5).
__device__ __forceinline__ bool is_huge(float m, float c) { return !(fabsf(m) * c < kHuge); }
__device__ __forceinline__ float base_of(float m, float c) { return m == -INFINITY ? 0.f : __fmul_rn(m, c); }
__device__ __forceinline__ float far_exponent(float x, float m, float c, float m_low = 0.f) {
  return ((x - (m == -INFINITY ? 0.f : m)) - m_low) * c;
}
__device__ __forceinline__ float exponent_of(float x, float m, float c) {
  return is_huge(m, c) ? far_exponent(x, m, c) : fmaf(x, c, -base_of(m, c));
}
// A sum against v.m, brought to a maximum m >= v.m: by the difference of the two
// bases as they were rounded (1 exactly where the maximum stays).
__device__ __forceinline__ float rebased(MaxSum v, float m, float c) {
  const float e = is_huge(m, c) ? far_exponent(v.m, m, c) : __fsub_rn(__fmul_rn(v.m, c), base_of(m, c));
  return v.s * ex2(e);
}

// The maximum over the lanes of a warp, in all of them (a NaN is passed over;
// the sum of exponentials then carries it).
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
// Sums over groups of W lanes, the same bits in all of them (each step adds the same two values).
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The pairs of W lanes (repeated over the warp) as one.
template <int W>
__device__ __forceinline__ MaxSum lanes_total(MaxSum v, float c) {
  const float m = warp_max(v.m);
  return {m, lanes_sum<W>(rebased(v, m, c))};
}

// Copies and stores under a predicate, at fixed offsets from one address: as
// `if` statements each of them became a branch with its own address arithmetic,
// together a third of the instructions of a row.
template <int OFF>
__device__ __forceinline__ void cp_async_16_if(bool p, uint32_t smem, const void* src) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
      "@p cp.async.cg.shared.global [%1 + %3], [%2 + %3], 16;\n\t}" ::"r"((int)p),
      "r"(smem), "l"(src), "n"(OFF)
      : "memory");
}
template <int OFF>
__device__ __forceinline__ void st_v2_if(bool p, void* dst, uint32_t a, uint32_t b) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p st.global.v2.b32 [%1 + %4], {%2, %3};\n\t}" ::"r"(
                   (int)p),
               "l"(dst), "r"(a), "r"(b), "n"(OFF)
               : "memory");
}
template <int OFF>
__device__ __forceinline__ void st_v4_if(bool p, void* dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p st.global.v4.b32 [%1 + %6], {%2, %3, %4, %5};\n\t}" ::"r"(
          (int)p),
      "l"(dst), "r"(a), "r"(b), "r"(c), "r"(d), "n"(OFF)
      : "memory");
}
// f(integral_constant<0>), f(integral_constant<1>), ...: a loop whose index is a constant
template <typename F, int... I>
__device__ __forceinline__ void unrolled(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

// A pair into another CTA's shared memory, counted (8 bytes) on a barrier there.
__device__ __forceinline__ void st_async_pair(uint32_t dst, MaxSum v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(dst), "f"(v.m),
               "f"(v.s), "r"(bar)
               : "memory");
}

// Two fp32 operations in one instruction: what is issued per logit counts.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ uint64_t ex2_2(uint64_t e) {
  const float2 f = unpair(e);
  return pair(ex2(f.x), ex2(f.y));
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

// A teacher entry: token id (-1: padding, its logit then -infinity) and logit.
struct Entry {
  int id;
  float t;
};
// As loaded: nothing waits for the loads before the entry is used, a row later.
struct RawEntry {
  int id;
  uint32_t bits;
};
__device__ __forceinline__ RawEntry load_entry(const DistillArgs& a, int m, int j) {
  const size_t at = (size_t)m * a.k + j;
  RawEntry e;
  e.id = a.indices[at];
  if (a.half_teacher) e.bits = static_cast<const unsigned short*>(a.teacher)[at];
  else e.bits = static_cast<const uint32_t*>(a.teacher)[at];
  return e;
}
__device__ __forceinline__ Entry entry_of(const DistillArgs& a, const RawEntry& e) {
  return {e.id, a.half_teacher ? __half2float(__ushort_as_half((unsigned short)e.bits)) : __uint_as_float(e.bits)};
}

// A step of two launches hands the log-sum-exp from the first to the second.  In
// fp32 that is good for p while the row is near zero (about 4 |lse| 2^-24 of p, at
// the limit 1.5e-5, a thirtieth of the fp16 rounding); of a row far from it the
// fraction is lost, and one that is masked whole by the lowest value would have p =
// 1 instead of 1 / V.  For such a row the first launch also leaves the pair itself,
// where the gradient of each tile will stand: only that tile's CTA reads it there,
// before it writes.  (A pair for every row: 2048 x 32000 in fp16 83.9 us instead of
// 81.6, 891 x 73496 264 instead of 261; none at all 81.4 and 256.)
constexpr float kNear = 64.f;
__device__ __forceinline__ bool is_near(float lse) { return fabsf(lse) < kNear; }
// The place for the tile that begins at vector `begin` (of E logits): 16-byte
// aligned, 8 logits at least.
__device__ __forceinline__ MaxSum* pair_of_tile(const DistillArgs& a, int m, int begin, int E) {
  return reinterpret_cast<MaxSum*>(a.grad + (size_t)m * a.V + (size_t)begin * E);
}

// Rows (kLoss, kStep): grid = clusters of C CTAs (a power of two); cluster q
// takes rows q, q + clusters, ...; CTA `rank` owns the vectors [rank VV / C, (rank
// + 1) VV / C) of each (VV = V / E), in `tiles` tiles (kStep: one, which stays in
// registers).  Gradient alone (kGrad): no clusters; CTA b takes items b, b + grid,
// ... of the M x C tiles.  Dynamic shared memory: the next tile, two sets of k
// teacher entries.
enum Mode { kLoss, kStep, kGrad };
// PAIR: the two launches of a step (a run-time branch cost the loss and the
// gradient alone 4 %).
template <int MODE, bool HALF, bool PAIR>
__global__ void __launch_bounds__(kThreads, kPerSm) q4gsw_distill_kernel(const DistillArgs a, int C, int tiles) {
  constexpr bool ROWS = MODE != kGrad, want_grad = MODE != kLoss;
  constexpr int E = HALF ? 8 : 4;         // logits per vector
  constexpr int NV = kPer / E;            // vectors per thread and tile
  constexpr int TV = kTile / E;           // vectors per tile
  extern __shared__ uint4 s_next[];       // [NV][kThreads]
  __shared__ MaxSum s_warp[kWarps];       // the warps' pairs
  __shared__ MaxSum s_row[2][kMaxCluster];   // the row's CTAs' pairs
  __shared__ MaxSum s_teach[2][kWarps];   // of the warps with entries; (-infinity, 0) from the others
  __shared__ float s_loss[kWarps];
  __shared__ uint64_t s_bar[2];
  __shared__ int s_abort;
  const int k = a.k, V = a.V;
  const int k4 = (k + 3) & ~3;                                         // ids in groups of four
  int* s_id = reinterpret_cast<int*>(s_next + NV * kThreads);          // [2][k4], -1: padding
  float* s_t = reinterpret_cast<float*>(s_id + 2 * k4);                // [2][k4]

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inv_t = a.inv_t, c = a.inv_t * kLog2e;
  const int VV = V / E;
  const int c_log = __ffs(C) - 1;
  const int rank = ROWS ? blockIdx.x & (C - 1) : 0;
  const int first = ROWS ? blockIdx.x >> c_log : blockIdx.x, step = ROWS ? gridDim.x >> c_log : gridDim.x;
  const int items = ROWS ? a.M : a.M * C;   // rows, or tiles of rows
  if (MODE != kLoss) tiles = 1;
  const bool entry_warp = 32 * warp < k;   // a warp whose threads have teacher entries

  // Vectors [begin, end) of row m.
  struct Span {
    int m, begin, end;
  };
  const int v_begin = ROWS ? (int)(((long long)rank * VV) >> c_log) : 0;
  const int v_end = ROWS ? (int)(((long long)(rank + 1) * VV) >> c_log) : 0;
  auto slice_of = [&](int it) -> Span {
    if (ROWS) return {it, v_begin, v_end};
    const int m = it / C, t = it - m * C;
    return {m, t * TV, min(VV, (t + 1) * TV)};
  };
  // vectors of load `l` of an item (a tile of the slice)
  auto span_of = [&](int it, int l) -> Span {
    Span s = slice_of(it);
    if (MODE == kLoss && tiles > 1) {
      s.begin += l * TV;
      s.end = min(s.end, s.begin + TV);
    }
    return s;
  };
  auto row_of = [&](int m) { return static_cast<const char*>(a.logits) + (size_t)m * V * (HALF ? 2 : 4); };
  // logits past the end of the slice: -infinity, which adds nothing
  const uint4 fill = HALF ? make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u)
                          : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  // Each thread copies, and later reads, its own vectors: no barrier.  They
  // are issued after the tile before has been consumed from registers.  Slots
  // past the end of a slice are filled once where all slices are alike.
  uint4* const slots = s_next + threadIdx.x;
  const uint32_t slots_addr = sm100::smem_u32(slots);
  auto issue = [&](const Span& s) {
    const uint4* src = reinterpret_cast<const uint4*>(row_of(s.m)) + s.begin + threadIdx.x;
    const int n = s.end - s.begin - (int)threadIdx.x;
    unrolled(
        [&](auto index) {
          constexpr int i = decltype(index)::value;
          cp_async_16_if<i * kThreads * 16>(i * kThreads < n, slots_addr, src);
        },
        std::make_integer_sequence<int, NV>{});
    cp_async_commit();
    if (MODE == kGrad || (MODE == kLoss && tiles > 1)) {
#pragma unroll 1
      for (int i = NV - 1; i >= 0 && i * kThreads >= n; --i) slots[i * kThreads] = fill;
    }
  };
  auto take = [&](uint4 (&x)[NV]) {
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = lds128_u32addr(slots_addr + i * kThreads * 16);
  };

  if (ROWS && tiles == 1) {
#pragma unroll 1
    for (int i = 0; i < NV; ++i)
      if (i * kThreads + (int)threadIdx.x >= v_end - v_begin) slots[i * kThreads] = fill;
  }
  if (threadIdx.x < 2 * kWarps) s_teach[threadIdx.x / kWarps][threadIdx.x % kWarps] = {-INFINITY, 0.f};
  if (threadIdx.x < kWarps) s_loss[threadIdx.x] = 0.f;
  __syncthreads();
  if (ROWS && C > 1) {
    if (threadIdx.x == 0) {
      sm100::mbar_init(&s_bar[0], 1);
      sm100::mbar_init(&s_bar[1], 1);
      s_abort = 0;
      sm100::fence_mbar_init();
    }
  }

  griddep_wait();
  RawEntry ahead{-1, 0u};      // entry threadIdx.x of the next item
  float d_loss_ahead = 0.f, lse_ahead = 0.f;
  auto fetch = [&](int m) {
    if ((int)threadIdx.x < k) ahead = load_entry(a, m, threadIdx.x);
    if (want_grad) d_loss_ahead = a.d_loss[m];
    if (!ROWS) lse_ahead = a.lse_in[m];
  };
  if (first < items) {
    const Span s = span_of(first, 0);
    issue(s);
    fetch(s.m);
  }
  if (ROWS && C > 1) sm100::cluster_barrier();   // every CTA's barriers are set up

  int turn = 0;   // items done
  for (int it = first; it < items; it += step, ++turn) {
    const int par = turn & 1;
    const Span slice = slice_of(it);
    const int m = slice.m;
    const char* row = row_of(m);
    const float coef = d_loss_ahead * a.temperature, lse_saved = lse_ahead;
    MaxSum mine{0.f, 1.f};    // the row's pair (kGrad: of a row far from zero)
    if (!ROWS && PAIR && !is_near(lse_saved)) mine = *pair_of_tile(a, m, slice.begin, E);
    int* ids = s_id + par * k4;
    float* ts = s_t + par * k4;

    // ---- teacher entries -> shared memory; the (max, sum) of the warp's
    bool some = false;            // an entry with a weight (a NaN counts as one)
    float z_own = 0.f;            // the student's logit at entry threadIdx.x, where this CTA needs it
    if (entry_warp) {
      float t_max = -INFINITY, t_sum = 0.f;
      for (int j = threadIdx.x; j < k4; j += kThreads) {
        Entry e{-1, -INFINITY};
        if (j < k) e = entry_of(a, j == (int)threadIdx.x ? ahead : load_entry(a, m, j));
        if (e.id < 0 || e.id >= V) {
          if (e.id != -1 && rank == 0) atomicOr(&g_device_error, kIndexErrorBit);
          e = {-1, -INFINITY};
        }
        ids[j] = e.id;
        ts[j] = e.t;
        some |= !(e.t == -INFINITY);
        if (j == (int)threadIdx.x && e.id >= 0 &&
            ((ROWS && rank == 0) || (e.id >= slice.begin * E && e.id < slice.end * E)))
          z_own = logit_at<HALF>(row, e.id);
        t_max = fmaxf(t_max, e.t);
      }
      t_max = warp_max(t_max);
      for (int j = threadIdx.x; j < k4; j += kThreads) t_sum += ex2(exponent_of(ts[j], t_max, c));   // its own entries
      t_sum = lanes_sum<32>(t_sum);
      if (lane == 0) s_teach[par][warp] = {t_max, t_sum};
    }

    // ---- (max, sum of exponentials) of the slice; run_m is the same in a warp
    uint4 x[NV];
    float run_m = -INFINITY, run_s = 0.f;
    if (ROWS) {
      for (int l = 0; l < tiles; ++l) {
        take(x);
        float top_t = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float f[E];
          unpack<HALF>(x[i], f);
#pragma unroll
          for (int e = 0; e < E; ++e) top_t = fmaxf(top_t, f[e]);
        }
        // every vector is in registers (the maximum depends on it): its slots take the next load
        const float mx = fmaxf(run_m, warp_max(top_t)), base = base_of(mx, c);
        if (l + 1 < tiles) issue(span_of(it, l + 1));
        else if (it + step < items) issue(span_of(it + step, 0));
        uint64_t sum[2] = {pair(rebased({run_m, run_s}, mx, c), 0.f), 0ull};
        const uint64_t c2 = pair(c, c), minus_base = pair(-base, -base);
        auto add = [&](auto weights) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            float f[E];
            unpack<HALF>(x[i], f);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const uint64_t w = weights(f[e], f[e + 1]);
              sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], w);
              const float2 kept = unpair(w);
              f[e] = kept.x;
              f[e + 1] = kept.y;
            }
            // the weights take the logits' registers: the gradient is a factor away from them
            if constexpr (MODE == kStep)
              x[i] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                __float_as_uint(f[3]));
          }
        };
        if (!is_huge(mx, c)) add([&](float z0, float z1) { return ex2_2(fma2(pair(z0, z1), c2, minus_base)); });
        else add([&](float z0, float z1) { return ex2_2(pair(far_exponent(z0, mx, c), far_exponent(z1, mx, c))); });
        const float2 total = unpair(add2(sum[0], sum[1]));
        run_m = mx;
        run_s = total.x + total.y;
      }
      run_s = lanes_sum<32>(run_s);
      if (lane == 0) s_warp[warp] = {run_m, run_s};
    } else {
      take(x);
    }
    if (it + step < items) fetch(slice_of(it + step).m);
    const bool has = __syncthreads_or(some);
    // No arithmetic has waited for this mode's reads of the slots yet: the barrier
    // has, so that the copies into them come after it.
    if (!ROWS && it + step < items) issue(span_of(it + step, 0));

    // ---- the row's pair: every CTA's to every CTA of the cluster
    if (ROWS) {
      mine = lanes_total<kWarps>(s_warp[lane % kWarps], c);
      if (C > 1 && warp == kWarps - 1) {
        if (lane == 0) sm100::mbar_arrive_expect_tx(&s_bar[par], (uint32_t)sizeof(MaxSum) * C);
        __syncwarp();
        if (lane < C)
          st_async_pair(sm100::mapa_u32(sm100::smem_u32(&s_row[par][rank]), lane), mine,
                        sm100::mapa_u32(sm100::smem_u32(&s_bar[par]), lane));
      }
    }
    MaxSum teach{0.f, 0.f};   // in the warps with entries
    float inv_total = 0.f;    // q_j = 2^exponent_of(t_j, teach.m) / teach.s
    if (entry_warp) {
      teach = lanes_total<kWarps>(s_teach[par][lane % kWarps], c);
      inv_total = 1.f / teach.s;
    }
    // p_i = 2^(z_i c - base) scale, base for ref; far from zero 2^((z_i - ref - ref_low) c) scale
    float ref, base, scale, ref_low = 0.f;
    bool far_lse = false;
    auto far = [&] { return ROWS ? is_huge(ref, c) : far_lse; };
    if (ROWS) {
      if (C > 1) {
        // (out of time: s_abort and the device error word are set, the row's results are not valid)
        sm100::mbar_wait(&s_bar[par], (turn >> 1) & 1, &s_abort, &g_device_error, 0x400u);
        mine = lane % kMaxCluster < C ? s_row[par][lane % kMaxCluster] : MaxSum{-INFINITY, 0.f};
        mine = lanes_total<kMaxCluster>(mine, c);
      }
      ref = mine.m;
      base = base_of(ref, c);
      scale = 1.f / mine.s;
      if (rank == 0 && entry_warp) {
        // log of the sum against the maximum itself (its base was rounded)
        auto log_of = [&](const MaxSum& v) {
          return logf(v.s) - (is_huge(v.m, c) ? 0.f : fmaf(v.m, c, -base_of(v.m, c)) * kLn2);
        };
        // (ref - ref) is 0, or NaN where the row's maximum is not finite
        const float log_sum = log_of(mine) + (ref - ref);
        float part = 0.f;
        if (has) {
          const float log_total = log_of(teach);
          for (int j = threadIdx.x; j < k; j += kThreads) {
            const Entry e{ids[j], ts[j]};
            const float q = ex2(exponent_of(e.t, teach.m, c)) * inv_total;
            // a weight of zero adds nothing, whatever its token's logit (a NaN weight is added)
            if (e.id >= 0 && !(q == 0.f)) {
              const float z = j == (int)threadIdx.x ? z_own : logit_at<HALF>(row, e.id);
              // both sides against their maxima: in lse itself a row far from zero has lost the
              // fraction of its logarithm (1e-3 of the loss at logits around 2e4)
              part += q * ((e.t - teach.m) * inv_t - log_total - (z - ref) * inv_t + log_sum);
            }
          }
        }
        part = lanes_sum<32>(part);
        if (lane == 0) s_loss[warp] = part;
        const float lse = fmaf(ref, inv_t, log_sum);
        if (threadIdx.x == 0) a.lse[m] = lse;
        if (MODE == kLoss && PAIR && warp == 0 && !is_near(lse))
          for (int v = lane * TV; v < VV; v += 32 * TV) *pair_of_tile(a, m, v, E) = mine;
      }
    } else if (PAIR && !is_near(lse_saved)) {
      ref = mine.m;
      base = base_of(ref, c);
      scale = 1.f / mine.s;
      far_lse = is_huge(ref, c);
    } else {
      // z / T - lse = (z - lse T) / T.  Here nothing cancels what rounding z c and the
      // base changed (4 |lse| 2^-24 of p): far from zero the difference comes first,
      // against lse T in two parts, and its rounding is one of the difference.
      ref = __fmul_rn(lse_saved, a.temperature);
      base = lse_saved * kLog2e;
      scale = 1.f;
      far_lse = !is_near(lse_saved);
      if (far_lse && fabsf(ref) < INFINITY) ref_low = fmaf(lse_saved, a.temperature, -ref);
    }

    // ---- gradient: coef p for every token of the slice, then the teacher's tokens again
    __half* grow = a.grad + (size_t)m * V;
    if (want_grad) {
      // the logits (kStep: their weights) stay as they are: unpacked early, those of
      // fp16 rows took twice the registers through the barriers, and spilled
#pragma unroll
      for (int i = 0; i < NV; ++i) asm volatile("" : "+r"(x[i].x), "+r"(x[i].y), "+r"(x[i].z), "+r"(x[i].w));
      // (kStep) the weights are against the warp's maximum
      const float by = coef * scale * (MODE == kStep ? rebased({run_m, 1.f}, ref, c) : 1.f);
      const uint64_t c2 = pair(c, c), minus_base = pair(-base, -base), by2 = pair(by, by);
      __half* dst = grow + ((size_t)slice.begin + threadIdx.x) * E;
      const int n = slice.end - slice.begin - (int)threadIdx.x;
      auto store = [&](auto values) {
        unrolled(
            [&](auto index) {
              constexpr int i = decltype(index)::value;
              float f[E];
              unpack<HALF>(x[i], f);
              uint32_t h[E / 2];
#pragma unroll
              for (int e = 0; e < E; e += 2) {
                const float2 g = unpair(values(f[e], f[e + 1]));
                h[e / 2] = h2_as_u32(__floats2half2_rn(g.x, g.y));
              }
              constexpr int kOff = i * kThreads * E * 2;
              if constexpr (HALF) st_v4_if<kOff>(i * kThreads < n, dst, h[0], h[1], h[2], h[3]);
              else st_v2_if<kOff>(i * kThreads < n, dst, h[0], h[1]);
            },
            std::make_integer_sequence<int, NV>{});
      };
      if (!has) store([&](float, float) { return 0ull; });
      else if (MODE == kStep) store([&](float w0, float w1) { return mul2(pair(w0, w1), by2); });
      else if (!far())
        store([&](float z0, float z1) { return mul2(ex2_2(fma2(pair(z0, z1), c2, minus_base)), by2); });
      else if (PAIR)   // rare: near the end of the fp32 range
        store([&](float z0, float z1) {
          return mul2(ex2_2(pair(far_exponent(z0, ref, c, ref_low), far_exponent(z1, ref, c, ref_low))), by2);
        });
      else {   // the same, two at a time (2048 x 32000 around 200: 57.7 us instead of 60.1; PAIR would spill)
        const float minus = ref == -INFINITY ? 0.f : -ref;
        const uint64_t minus_ref = pair(minus, minus), minus_low = pair(-ref_low, -ref_low);
        store([&](float z0, float z1) {
          return mul2(ex2_2(mul2(add2(add2(pair(z0, z1), minus_ref), minus_low), c2)), by2);
        });
      }
    }
    __syncthreads();
    if (ROWS && rank == 0 && threadIdx.x == 0) {
      float sum = 0.f;
      for (int w = 0; w < kWarps; ++w) sum += s_loss[w];   // 0 from the warps without entries
      a.loss[m] = sum * a.temperature * a.temperature;
    }
    if (want_grad && has && entry_warp) {
      for (int j = threadIdx.x; j < k; j += kThreads) {
        const int id = ids[j];
        if (id < slice.begin * E || id >= slice.end * E) continue;   // padding, or another CTA's token
        const float z = j == (int)threadIdx.x ? z_own : logit_at<HALF>(row, id);
        int same = 0;
        for (int q = 0; q < k4; q += 4) {
          const int4 o = *reinterpret_cast<const int4*>(ids + q);
          same += (o.x == id) + (o.y == id) + (o.z == id) + (o.w == id);
        }
        float t = ex2(exponent_of(ts[j], teach.m, c));
        if (same > 1) {   // every entry of this token, in the order of the list: each of them writes the same value
          t = 0.f;
          for (int q = 0; q < k; ++q)
            if (ids[q] == id) t += ex2(exponent_of(ts[q], teach.m, c));
        }
        const float p = ex2(far() ? far_exponent(z, ref, c, ref_low) : fmaf(z, c, -base)) * scale;
        grow[id] = __float2half_rn(coef * (p - t * inv_total));
      }
    }
    if (ROWS && C > 1 && *static_cast<volatile int*>(&s_abort)) {
      // A wait of this row ran out.  Every warp sees it, since a barrier stands
      // before the next wait, so all of them leave with the same row.  A peer may
      // still be on its way to this row and then writes its pair here: stay until
      // every CTA of the cluster has left or stands here too (their waits are as
      // bounded as this one was).
      sm100::cluster_barrier();
      break;
    }
  }
  cp_async_wait<0>();   // nothing in flight when a wait ran out
}

}  // namespace distill

// Launch configuration of clusters of C (ROWS) or single CTAs.
struct DistillConfig {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  DistillConfig(unsigned grid, int C, bool rows, size_t smem, cudaStream_t stream) {
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(distill::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = rows ? 2 : 1;
  }
  DistillConfig(const DistillConfig&) = delete;
};

// One instance: a mode, fp16 or fp32 logits, whether a pair per row goes from launch to launch.
template <int MODE, bool HALF, bool PAIR>
struct DistillKernel {
  static auto kernel() { return distill::q4gsw_distill_kernel<MODE, HALF, PAIR>; }

  // bytes of the next tile, two sets of k teacher entries
  static size_t smem(int k) { return (size_t)distill::kTile * (HALF ? 2 : 4) + (size_t)((k + 3) & ~3) * 16; }

  static cudaError_t setup() {
    static PerDeviceOnce attr_once;
    return once_per_device(attr_once, current_device(), [] {
      const cudaError_t e = cudaFuncSetAttribute(kernel(), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem(1024));
      return e != cudaSuccess ? e : cudaFuncSetAttribute(kernel(), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
  }

  static cudaError_t launch(const DistillArgs& a, int C, int tiles, unsigned grid, cudaStream_t stream) {
    const cudaError_t e = setup();
    if (e != cudaSuccess) return e;
    DistillConfig c(grid, C, MODE != distill::kGrad, smem(a.k), stream);
    return cudaLaunchKernelEx(&c.cfg, kernel(), a, C, tiles);
  }

  // Clusters of C CTAs the current device holds at once (asked once per device,
  // for teacher lists of up to 256 entries and for longer ones).
  static int clusters(int C, int k) {
    static std::atomic<int> cached[kMaxDevices][2][distill::kMaxCluster + 1];
    const int dev = current_device();
    const int d = (dev >= 0 && dev < kMaxDevices) ? dev : 0, big = k > 256;
    int n = cached[d][big][C].load(std::memory_order_relaxed);
    if (n == 0) {
      n = -1;
      if (setup() == cudaSuccess) {
        DistillConfig c((unsigned)C, C, true, smem(big ? 1024 : 256), nullptr);
        if (cudaOccupancyMaxActiveClusters(&n, kernel(), &c.cfg) != cudaSuccess || n < 1) n = -1;
      }
      cached[d][big][C].store(n, std::memory_order_relaxed);
    }
    return n > 0 ? n : 1;
  }
};

template <int MODE, bool HALF, bool PAIR>
static cudaError_t distill_rows(const DistillArgs& a, cudaStream_t stream, char* route, int route_len) {
  using namespace distill;
  // CTAs per row.  The loss alone needs no row held: one CTA walks it, unless
  // the rows are too few to fill the SMs (702 x 93232 in fp16: two CTAs a row
  // 30 us, 16 of a single tile each 101: a row's fixed work, its reductions and
  // the teacher's list, is then done for ever smaller slices).  With a gradient, as
  // many as hold the row.  Both grow, down to 2048 logits a CTA, while CTAs are
  // idle.
  const int sms = sm_count(current_device());
  int C = 1;
  if (MODE == kStep)
    while (C < kHoldCluster && (long long)C * kTile < a.V) C *= 2;
  while (C < kMaxCluster && (long long)a.M * C < (MODE == kStep ? sms : kPerSm * sms) && a.V / (2 * C) >= 2048) C *= 2;
  const int E = HALF ? 8 : 4;
  const int tiles = (int)(((a.V / E + C - 1LL) / C * E + kTile - 1) / kTile);   // (V may end at 2^31 - 8)
  // one wave of clusters (a cluster that had to wait for a slot would start its
  // rows when the others end theirs)
  const int most = DistillKernel<MODE, HALF, PAIR>::clusters(C, a.k);
  const unsigned n = (unsigned)(a.M < most ? a.M : most);
  if (route)
    snprintf(route, route_len, "distill_%s launches=1 cluster=%d clusters=%u tiles=%d", MODE == kStep ? "step" : "fwd", C, n,
             tiles);
  return DistillKernel<MODE, HALF, PAIR>::launch(a, C, tiles, n * C, stream);
}

template <bool HALF, bool PAIR>
static cudaError_t distill_grad(const DistillArgs& a, cudaStream_t stream, char* route, int route_len) {
  using namespace distill;
  const int C = (a.V - 1) / kTile + 1;   // (V may end at 2^31 - 8)
  const long long items = (long long)a.M * C;
  const int most = kPerSm * sm_count(current_device());
  const unsigned grid = (unsigned)(items < most ? items : most);
  if (route) snprintf(route, route_len, "distill_bwd launches=1 tiles=%d ctas=%u", C, grid);
  return DistillKernel<kGrad, HALF, PAIR>::launch(a, C, 1, grid, stream);
}

cudaError_t launch_distill_bwd(const DistillArgs& a, bool half_logits, cudaStream_t stream, char* route,
                               int route_len) {
  return half_logits ? distill_grad<true, false>(a, stream, route, route_len)
                     : distill_grad<false, false>(a, stream, route, route_len);
}

// The loss, then the gradient.
template <bool HALF>
static cudaError_t distill_step_in_two(DistillArgs a, cudaStream_t stream, char* route, int route_len) {
  const cudaError_t e = distill_rows<distill::kLoss, HALF, true>(a, stream, nullptr, 0);
  if (e != cudaSuccess) return e;
  if (route) snprintf(route, route_len, "distill_step launches=2 fwd + bwd");
  a.lse_in = a.lse;
  return distill_grad<HALF, true>(a, stream, nullptr, 0);
}

cudaError_t launch_distill_rows(const DistillArgs& a, bool half_logits, cudaStream_t stream, char* route,
                                int route_len) {
  using namespace distill;
  // Loss and gradient in one pass for fp32 logits while a cluster of eight holds
  // the row and the teacher's list is short.  Otherwise the loss, then the
  // gradient.  Measured (us, one pass and two): 512 x 32000 with k = 64 25 and 36;
  // 891 x 73496 with k = 319 317 and 169; fp16 logits, which two passes move in 6
  // bytes instead of 4, 2048 x 32000 84 and 78.
  if (a.grad && (half_logits || a.V > kHoldCluster * kTile || a.k > kThreads))
    return half_logits ? distill_step_in_two<true>(a, stream, route, route_len)
                       : distill_step_in_two<false>(a, stream, route, route_len);
  if (a.grad) return distill_rows<kStep, false, false>(a, stream, route, route_len);
  return half_logits ? distill_rows<kLoss, true, false>(a, stream, route, route_len)
                     : distill_rows<kLoss, false, false>(a, stream, route, route_len);
}

}  // namespace q4gsw
