// Clipped policy loss with a KL term, forward and backward from the logits.
//
// With z = logits / temperature, y the row's target and w its weight:
//   logp = z_y - log sum exp z,  r = exp(logp - old),  A the advantage
//   row  = -min(r A, clip(r, 1 - lo, 1 + hi) A) + b (exp(d) - d - 1),  d = ref - logp
//   loss = sum_rows w row
//   dlogits = grad_scale w c / temperature (onehot(y) - softmax z),
//   c = d row / d logp = -A r [r A <= clip(r) A] + b (1 - exp(d))
#include <cooperative_groups.h>

#include "train_common.cuh"

namespace ftmoe {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;  // 16-byte loads a thread has in flight
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A running maximum of logits and the sum of 2^(k2 (x - maximum)), k2 =
// log2(e) / temperature.  The maximum is subtracted before the product: a
// fused x k2 - m k2 would leave the rounding of m k2 in every exponent, which
// for logits near the type's lowest value is itself large.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float k2) {
  const float m = fmaxf(a.m, b.m), ref = m == -INFINITY ? 0.f : m;
  return {m, a.s * exp2_fast((a.m - ref) * k2) + b.s * exp2_fast((b.m - ref) * k2)};
}

// One row's 16-byte pieces.  The row starts `skip` values after a 16-byte
// boundary; the first and the last piece may belong to it in part, and are
// then read and written value by value.
template <typename T>
struct Row {
  static constexpr int N = 16 / sizeof(T);
  T* at;  // the boundary
  int skip;
  int64_t end;  // skip + V
  __device__ Row(const T* p, int64_t V) {
    skip = (int)(((uintptr_t)p & 15) / sizeof(T));
    at = const_cast<T*>(p) - skip;
    end = skip + V;
  }
  __device__ int64_t pieces() const { return (end + N - 1) / N; }
  __device__ bool whole(int64_t i) const { return i * N >= skip && (i + 1) * N <= end; }
  __device__ Pack<T, N> load(int64_t i) const {
    if (whole(i)) return load_pack<T, N>(at + i * N);
    Pack<T, N> r;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int64_t e = i * N + c;
      r.set(c, -INFINITY);
      if (e >= skip && e < end) r.v[c] = at[e];
    }
    return r;
  }
  __device__ void store(int64_t i, const Pack<T, N>& r, bool same) const {
    if (same && whole(i)) {
      store_pack<T, N>(at + i * N, r);
      return;
    }
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int64_t e = i * N + c;
      if (e >= skip && e < end) at[e] = r.v[c];
    }
  }
};

// A cluster takes a row, each CTA a contiguous part of its pieces.  STAGED:
// the part stays in shared memory between the softmax's sum and the gradient.
template <typename T, bool STAGED>
__global__ void __launch_bounds__(kThreads) k_policy(ftmoe_policy_args a, uint32_t* status) {
  extern __shared__ __align__(16) unsigned char policy_smem[];
  __shared__ MaxSum warp_part[kWarps];
  __shared__ MaxSum exchange[2];
  constexpr int N = Row<T>::N;
  Pack<T, N>* stage = reinterpret_cast<Pack<T, N>*>(policy_smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float k2 = kLog2e / a.temperature;
  int parity = 0;
  for (int64_t n = blockIdx.x / ranks; n < a.N; n += gridDim.x / ranks) {
    const int64_t y = a.id_bytes == 8 ? static_cast<const int64_t*>(a.targets)[n]
                                      : static_cast<const int32_t*>(a.targets)[n];
    float w = a.weight ? a.weight[n] : 1.f / (float)a.N;
    const bool valid = y >= 0 && y < a.V;
    if (!valid && rank == 0 && tid == 0) set_status(status, kStatusRange);
    if (!valid) w = 0.f;
    const Row<T> z(static_cast<const T*>(a.logits) + n * a.ld, a.V);
    const int64_t per = (z.pieces() + ranks - 1) / ranks, lo = rank * per, hi = min(z.pieces(), lo + per);
    float c = 0.f, m = 0.f, ls = 0.f;  // the gradient's coefficient; softmax z = 2^((x - m) k2 - ls)
    if (w != 0.f) {
      const float zy = to_f32(z.at[z.skip + y]);
      MaxSum run{-INFINITY, 0.f};
      for (int64_t i0 = lo + tid; i0 < hi; i0 += kThreads * kAhead) {
        Pack<T, N> x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (i0 + u * kThreads < hi) x[u] = z.load(i0 + u * kThreads);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (i0 + u * kThreads >= hi) break;
          if (STAGED) stage[i0 + u * kThreads - lo] = x[u];
          float top = x[u].get(0);
#pragma unroll
          for (int e = 1; e < N; ++e) top = fmaxf(top, x[u].get(e));
          top = fmaxf(run.m, top);
          const float ref = top == -INFINITY ? 0.f : top;
          float s = run.s * exp2_fast((run.m - ref) * k2);
#pragma unroll
          for (int e = 0; e < N; ++e) s += exp2_fast((x[u].get(e) - ref) * k2);
          run = {top, s};
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        run = join(run, {__shfl_xor_sync(0xffffffffu, run.m, o), __shfl_xor_sync(0xffffffffu, run.s, o)}, k2);
      if (lane == 0) warp_part[warp] = run;
      __syncthreads();
      if (warp == 0) {
        run = lane < kWarps ? warp_part[lane] : MaxSum{-INFINITY, 0.f};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          run = join(run, {__shfl_xor_sync(0xffffffffu, run.m, o), __shfl_xor_sync(0xffffffffu, run.s, o)}, k2);
        if (lane == 0) exchange[parity] = run;
      }
      // Two exchange slots suffice: a CTA writes this one again two rows on,
      // and by then every peer has passed the next row's barrier, after its reads here.
      cluster.sync();
      run = lane < ranks ? *cluster.map_shared_rank(&exchange[parity], lane) : MaxSum{-INFINITY, 0.f};
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        run = join(run, {__shfl_xor_sync(0xffffffffu, run.m, o), __shfl_xor_sync(0xffffffffu, run.s, o)}, k2);
      parity ^= 1;
      m = run.m;
      ls = log2f(run.s);
      const float logp = ((zy - m) * k2 - ls) * kLn2;
      const float r = expf(logp - a.old_logp[n]), A = a.advantage[n];
      const float bounded = r < 1.f - a.clip_low ? 1.f - a.clip_low : r > 1.f + a.clip_high ? 1.f + a.clip_high : r;
      const bool clipped = r * A > bounded * A;  // false for NaN, which then reaches the loss and the gradient
      float row = -(clipped ? bounded * A : r * A);
      c = clipped ? 0.f : -(A * r);
      if (a.ref_logp && a.kl_coef != 0.f) {
        const float d = a.ref_logp[n] - logp, ed = expf(d);
        row += a.kl_coef * (ed - d - 1.f);
        c += a.kl_coef * (1.f - ed);
      }
      if (rank == 0 && tid == 0) {
        a.row_loss[n] = row;
        if (a.logp) a.logp[n] = logp;
      }
      c *= a.grad_scale * w / a.temperature;
    } else if (rank == 0 && tid == 0) {
      a.row_loss[n] = 0.f;
      if (a.logp) a.logp[n] = 0.f;
    }
    if (!a.dlogits) continue;
    const Row<T> g(static_cast<T*>(a.dlogits) + n * a.ld_d, a.V);
    const bool same = g.skip == z.skip;
    // a gradient row of another alignment is written value by value, at the logits' pieces
    const Row<T> out = [&] {
      Row<T> o = g;
      o.at += g.skip - z.skip;
      o.skip = z.skip;
      o.end = z.end;
      return o;
    }();
    if (c == 0.f) {  // nothing of the row's softmax is needed
      Pack<T, N> zero;
#pragma unroll
      for (int e = 0; e < N; ++e) zero.set(e, 0.f);
      for (int64_t i = lo + tid; i < hi; i += kThreads) out.store(i, zero, same);
      continue;
    }
    const int64_t target = z.skip + y;
    for (int64_t i0 = lo + tid; i0 < hi; i0 += kThreads * kAhead) {
      Pack<T, N> x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i0 + u * kThreads < hi) x[u] = STAGED ? stage[i0 + u * kThreads - lo] : z.load(i0 + u * kThreads);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t i = i0 + u * kThreads;
        if (i >= hi) break;
        Pack<T, N> o;
#pragma unroll
        for (int e = 0; e < N; ++e)
          o.set(e, c * ((i * N + e == target ? 1.f : 0.f) - exp2_fast(fmaf(x[u].get(e) - m, k2, -ls))));
        out.store(i, o, same);
      }
    }
  }
  cluster.sync();  // no CTA leaves while a peer may still read its exchange slot
}

// loss = sum_n w_n row_n in a fixed order, by one CTA.
__global__ void __launch_bounds__(1024) k_policy_sum(const float* weight, const float* row_loss, int64_t N, float* loss) {
  __shared__ double part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double s = 0.0;
  for (int64_t n = threadIdx.x; n < N; n += 1024) s += (double)(weight ? weight[n] : 1.f / (float)N) * row_loss[n];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) part[warp] = s;
  __syncthreads();
  if (warp == 0) {
    s = part[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) *loss = (float)s;
  }
}

// Shared memory a CTA may stage a part of a row in, and what lets three CTAs share an SM.
constexpr int kStageMax = 208 * 1024, kStageShared = 72 * 1024;
constexpr int kMaxRanks = 8;

}  // namespace

cudaError_t policy_set_limits() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto type) {
    return cudaFuncSetAttribute(k_policy<decltype(type), true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMax);
  };
  for (int t : {FTMOE_BF16, FTMOE_FP32, FTMOE_FP16})
    if ((e = with_dtype(t, set)) != cudaSuccess) return e;
  return e;
}

cudaError_t launch_policy_loss(const TrainDevice& d, const ftmoe_policy_args& a, cudaStream_t s) {
  if (a.N > 0) {
    const int bytes = dtype_bytes(a.dtype);
    const int64_t pieces = (a.V * bytes + 15 + 14) / 16 + 1;  // of a row at any alignment, at most
    auto part = [&](int ranks) { return (pieces + ranks - 1) / ranks * 16; };
    int ranks = 1;
    while (ranks < kMaxRanks && part(ranks) > kStageShared) ranks *= 2;
    // few rows: spread each over more CTAs while the SMs are not full and a part has work for its threads
    while (ranks < kMaxRanks && a.N * ranks < 2 * d.num_sms && part(ranks) >= 2 * kThreads * 16) ranks *= 2;
    const bool staged = a.dlogits && part(ranks) <= kStageMax;
    cudaLaunchConfig_t c{};
    const int64_t clusters = a.N < (1 << 24) ? a.N : (1 << 24);
    c.gridDim = dim3((unsigned)(clusters * ranks));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = staged ? (size_t)part(ranks) : 0;
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
    cudaError_t e = with_dtype(a.dtype, [&](auto type) {
      using T = decltype(type);
      return staged ? cudaLaunchKernelEx(&c, k_policy<T, true>, a, d.status)
                    : cudaLaunchKernelEx(&c, k_policy<T, false>, a, d.status);
    });
    if (e != cudaSuccess) return e;
  }
  k_policy_sum<<<1, 1024, 0, s>>>(a.weight, a.row_loss, a.N, a.loss);
  return cudaGetLastError();
}

}  // namespace ftmoe
