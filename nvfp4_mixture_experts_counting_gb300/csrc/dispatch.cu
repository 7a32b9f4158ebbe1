// Tokens sorted by expert and back: the dispatch (stable sort of the (token,
// slot) pairs by expert and the copy of each token's row to its sorted
// places), the weighted combine, and their gradients down to the router's logits.
//
// Pair p = t * k + j has expert e_p; a pair whose index is outside [0, E) is
// dropped.  offsets[e] = #{p : e_p < e}, and a kept pair's place is
// inv[p] = offsets[e_p] + #{q < p : e_q = e_p}.
#include <algorithm>
#include <type_traits>

#include "cluster_sort.cuh"

namespace ftmoe {

namespace {

constexpr int kThreads = 256;
// Pairs up to which every CTA counts its own tokens' places (one launch): at
// 2048 pairs that takes 4.5 us with the copy, the sort 4.4 us without it; at 4096 7.5 and 4.5 us.
constexpr int kCountPairs = 2048;
constexpr int kSlots = 4;      // slots of the combine that a thread has in flight
constexpr int kBackSlots = 8;  // and of its gradient

struct DispatchArgs {
  const int32_t* idx;
  int T, k, E, P;
  int32_t *offsets, *perm, *inv;
  uint32_t* status;
};

// offsets from a histogram of the experts; perm's places past the last kept pair become -1.
__device__ void dispatch_tables(const DispatchArgs& a) {
  __shared__ int hist[kMaxBins];
  __shared__ int wsum[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int e = tid; e < kMaxBins; e += kThreads) hist[e] = 0;
  __syncthreads();
  bool bad = false;
  for (int p = tid; p < a.P; p += kThreads) {
    const int e = a.idx[p];
    if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
    bad |= e >= a.E;
  }
  if (bad) set_status(a.status, kStatusRange);
  __syncthreads();
  constexpr int kPer = kMaxBins / kThreads;
  int v[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    v[i] = sum;
    sum += hist[tid * kPer + i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int before = 0, kept = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    before += w < warp ? wsum[w] : 0;
    kept += wsum[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e <= a.E) a.offsets[e] = before + inc - sum + v[i];
  }
  if (tid == 0 && a.E == kMaxBins) a.offsets[a.E] = kept;
  for (int p = kept + tid; p < a.P; p += kThreads) a.perm[p] = -1;
}

// Few pairs: one launch.  CTA t counts the places of token t's slots itself
// (a warp per slot reads all P indices; e_q < e_p + [q < p] is the test for
// "sorts before", and as unsigned values dropped pairs never pass it), then
// copies the row.  The first CTA writes the tables.  Latency bounds it: 2.6 us at
// T=16 k=8 H=2560 bf16, of which a launch takes 1.7.
template <int B>
__global__ void __launch_bounds__(kThreads) k_dispatch_count(DispatchArgs a, const void* x, int nv, void* xs) {
  using V = typename Raw<B>::type;
  const int t = (int)blockIdx.x - 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (t < 0) {
    dispatch_tables(a);
    return;
  }
  __shared__ int place[32];
  const V* src = static_cast<const V*>(x) + (int64_t)t * nv;
  V* dst = static_cast<V*>(xs);
  V row{};
  if (x && tid < nv) row = src[tid];
  for (int j = warp; j < a.k; j += kThreads / 32) {
    const int p = t * a.k + j, e = a.idx[p];
    const bool kept = e >= 0 && e < a.E;
    int n = 0;
    auto count = [&](int q, int other) { n += (unsigned)other < (unsigned)(e + (q < p ? 1 : 0)); };
    int q = 0;
    if (((uintptr_t)a.idx & 15) == 0) {
      const int4* four = reinterpret_cast<const int4*>(a.idx);
#pragma unroll 4
      for (; q + 128 <= a.P; q += 128) {
        const int4 v = four[q / 4 + lane];
        const int at = q + lane * 4;
        count(at, v.x);
        count(at + 1, v.y);
        count(at + 2, v.z);
        count(at + 3, v.w);
      }
    }
    for (q += lane; q < a.P; q += 32) count(q, a.idx[q]);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
      place[j] = kept ? n : -1;
      a.inv[p] = kept ? n : -1;
      if (kept) a.perm[n] = p;
    }
  }
  if (!x) return;
  __syncthreads();
  for (int v = tid; v < nv; v += kThreads) {
    if (v >= kThreads) row = src[v];
    for (int j = 0; j < a.k; ++j) {
      const int at = place[j];
      if (at >= 0) dst[(int64_t)at * nv + v] = row;
    }
  }
}

// Many pairs: the sort, by one cluster.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) k_dispatch_sort(DispatchArgs a) {
  extern __shared__ int sort_smem[];
  pdl_launch_dependents();
  bool bad = false;
  const int placed = cluster_sort<THREADS>(
      a.P, a.E, sort_smem, true,
      [&](int64_t i) {
        const int e = a.idx[i];
        bad |= e >= a.E;
        return SortItem{e, 0};
      },
      [&](int e) { return e < a.E ? e : -1; },
      [&](int64_t i, SortItem, int at) {
        a.inv[i] = at;
        if (at >= 0) a.perm[at] = (int)i;
      },
      [&](int e, int at) { a.offsets[e] = at; });
  if (bad) set_status(a.status, kStatusRange);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = placed;
  for (int64_t p = placed + (int64_t)blockIdx.x * THREADS + threadIdx.x; p < a.P; p += (int64_t)gridDim.x * THREADS)
    a.perm[p] = -1;
}

// ... and the copy: each thread reads Q pieces of a token's row, nq apart, and
// writes them to the row's k places.  Bound by the writes: T=16384 k=8 H=2560
// bf16 110 us, 6.9 TB/s.  The rows are asked for before the sort is done.
template <int B, int Q>
__global__ void __launch_bounds__(kThreads) k_dispatch_copy(const void* x, int64_t total, int nv, int nq, int k,
                                                            const int32_t* inv, void* xs) {
  using V = typename Raw<B>::type;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const int64_t t = quotient(i, nq);
  const int v = (int)(i - t * nq);
  V row[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q)
    if (v + q * nq < nv) row[q] = static_cast<const V*>(x)[t * nv + v + q * nq];
  V* dst = static_cast<V*>(xs) + v;
  pdl_wait();  // inv is the sort's
  for (int j = 0; j < k; ++j) {
    const int at = inv[t * k + j];
    if (at < 0) continue;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (v + q * nq < nv) dst[(int64_t)at * nv + q * nq] = row[q];
  }
}

// A pair's place, -1 if it is dropped or out of range.
__device__ __forceinline__ int checked_place(int at, int64_t P, uint32_t* status) {
  if (at < -1 || at >= P) {
    set_status(status, kStatusRange);
    return -1;
  }
  return at;
}

// out[t] = sum_j w[t, j] ys[inv[t, j]], slots in order, fp32.  A thread takes Q
// pieces of the row, nq apart, and kSlots slots at a time, whose loads are
// issued together: a slot that is dropped or past the last one has its
// neighbour's row loaded again and not used, as a load under a condition waits
// for the condition (bf16 T=16384 k=8 H=2560 took 386 us so).  Rows are read at the
// copy rate with many warps an SM: 48 with weights (111 us; 64 take 125, 40 take
// 136), 64 without (111 us; 48 take 122), where the 16-bit types spill 8 bytes.
template <typename T, int N, int Q, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads, N == 1 ? 1 : WEIGHTED ? 6 : 8)
    k_combine(const T* ys, int64_t total, int nv, int nq, int k, int64_t P, const int32_t* inv, const float* w, T* out,
              uint32_t* status) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const int64_t t = quotient(i, nq);
  const int v = (int)(i - t * nq);
  int at_column[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) at_column[q] = min(v + q * nq, nv - 1);
  float acc[Q][N] = {};
  for (int j0 = 0; j0 < k; j0 += kSlots) {
    Pack<T, N> y[kSlots][Q];
    int at[kSlots], some = 0;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      at[j] = j0 + j < k ? checked_place(inv[t * k + j0 + j], P, status) : -1;
      some = max(some, at[j]);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const T* row = ys + (int64_t)(at[j] < 0 ? some : at[j]) * nv * N;
#pragma unroll
      for (int q = 0; q < Q; ++q) y[j][q] = load_pack<T, N>(row + (int64_t)at_column[q] * N);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      if (at[j] < 0) continue;
      const float wj = WEIGHTED ? w[t * k + j0 + j] : 1.f;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
#pragma unroll
        for (int c = 0; c < N; ++c) acc[q][c] = fmaf(wj, y[j][q].get(c), acc[q][c]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (v + q * nq >= nv) break;
    Pack<T, N> o;
#pragma unroll
    for (int c = 0; c < N; ++c) o.set(c, acc[q][c]);
    store_pack<T, N>(out + (t * nv + v + q * nq) * N, o);
  }
}

// dys[inv[p]] = w[p] dout[t], dw[p] = <dout[t], ys[inv[p]]>: W warps take a
// token's row, kBackSlots slots at a time, whose loads are issued together (as
// in k_combine).  dys may be ys: a thread reads an element before it writes it,
// and no other thread uses it.  Every byte moves once: T=16384 k=8 H=2560 bf16
// 211 us, 6.8 TB/s, with 24 warps an SM (four slots and 32 warps: 239 us).
template <typename T, int N, int Q, int W>
__global__ void __launch_bounds__(kThreads, 3)
    k_combine_backward(const T* dout, const T* ys, int T_, int nv, int k, int64_t P, const int32_t* inv, const float* w,
                       T* dys, float* dw, uint32_t* status) {
  __shared__ float part[kThreads / 32][kBackSlots];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % W;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 32 / W) + warp / W;
  const bool on = t < T_;
  if (W == 1 && !on) return;
  for (int j0 = 0; j0 < k; j0 += kBackSlots) {
    int at[kBackSlots], some = 0;
    float wj[kBackSlots], dot[kBackSlots];
#pragma unroll
    for (int j = 0; j < kBackSlots; ++j) {
      const bool use = on && j0 + j < k;
      at[j] = use ? checked_place(inv[t * k + j0 + j], P, status) : -1;
      wj[j] = use ? w[t * k + j0 + j] : 0.f;
      dot[j] = 0.f;
      some = max(some, at[j]);
    }
    for (int v = sub * 32 * Q + lane; on && v < nv; v += 32 * Q * W) {
      Pack<T, N> d[Q], y[kBackSlots][Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) d[q] = load_pack<T, N>(dout + (t * nv + min(v + q * 32, nv - 1)) * N);
#pragma unroll
      for (int j = 0; j < kBackSlots; ++j) {
        const T* row = ys + (int64_t)(at[j] < 0 ? some : at[j]) * nv * N;
#pragma unroll
        for (int q = 0; q < Q; ++q) y[j][q] = load_pack<T, N>(row + (int64_t)min(v + q * 32, nv - 1) * N);
      }
#pragma unroll
      for (int j = 0; j < kBackSlots; ++j) {
        if (at[j] < 0) continue;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          if (v + q * 32 >= nv) break;
          Pack<T, N> o;
#pragma unroll
          for (int c = 0; c < N; ++c) {
            dot[j] = fmaf(d[q].get(c), y[j][q].get(c), dot[j]);
            o.set(c, wj[j] * d[q].get(c));
          }
          store_pack<T, N>(dys + ((int64_t)at[j] * nv + v + q * 32) * N, o);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBackSlots; ++j) dot[j] = warp_sum_f32(dot[j]);
    if (W > 1) {
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < kBackSlots; ++j) part[warp][j] = dot[j];
      }
      __syncthreads();
      if (on && sub == 0 && lane < kBackSlots && j0 + lane < k) {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < W; ++q) sum += part[warp + q][lane];
        dw[t * k + j0 + lane] = sum;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int j = 0; j < kBackSlots; ++j)
        if (lane == j && j0 + j < k) dw[t * k + j0 + j] = dot[j];
    }
  }
}

// The router's gradient, a warp per token.  With S = sum_j w_j dw_j,
//   renormalised weights:   dlogits[e] = sum_{j : idx_j = e} w_j (dw_j - S)
//   full-softmax weights:   dlogits[e] = p_e (sum_{j : idx_j = e} dw_j - S)
// The row is first written as if no expert were chosen (zeros, or -p_e S),
// then the chosen experts' values over it, each by the lane of its first slot
// (T=16384 E=256 k=8: 4.6 us renormalised; every expert compared with every slot
// took 12.  Full softmax 10.8 us: it reads the row three times and takes its
// exponentials twice).
template <bool NORM, int N>
__global__ void __launch_bounds__(kThreads) k_route_backward(const float* logits, const int32_t* idx, const float* w,
                                                             const float* dw, int T, int E, int k, float* dlogits,
                                                             uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (t >= T) return;
  const float* z = logits + t * E;
  float* out = dlogits + t * E;
  int ej = -1;
  float wj = 0.f, dj = 0.f;
  if (lane < k) {
    ej = idx[t * k + lane];
    wj = w[t * k + lane];
    dj = dw[t * k + lane];
    if (ej < 0 || ej >= E) {
      set_status(status, kStatusRange);
      ej = -1;
    }
  }
  const float zj = !NORM && ej >= 0 ? z[ej] : 0.f;  // before the row is written: dlogits may be the logits
  const float S = warp_sum_f32(wj * dj);
  const float up = NORM ? wj * (dj - S) : dj;
  float top = 0.f, sum = 1.f;
  if (!NORM) {
    top = -INFINITY;
    for (int e = lane; e < E; e += 32) top = fmaxf(top, z[e]);
    top = warp_max_f32(top);
    sum = 0.f;
    for (int e = lane; e < E; e += 32) sum += expf(z[e] - top);
    sum = warp_sum_f32(sum);
  }
  for (int e = lane * N; e < E; e += 32 * N) {
    Pack<float, N> o;
#pragma unroll
    for (int c = 0; c < N; ++c) o.v[c] = NORM ? 0.f : expf(z[e + c] - top) / sum * -S;
    store_pack<float, N>(out + e, o);
  }
  // slots of one expert (a router chooses distinct ones, a caller need not) share a sum
  float g = 0.f;
  bool first = true;
  for (int j = 0; j < k; ++j) {
    const int other = __shfl_sync(0xffffffffu, ej, j);
    const float u = __shfl_sync(0xffffffffu, up, j);
    if (other == ej) {
      g += u;
      first = first && j >= lane;
    }
  }
  __syncwarp();  // the row's first values are written
  if (lane < k && ej >= 0 && first) out[ej] = NORM ? g : expf(zj - top) / sum * (g - S);
}

inline unsigned blocks_of(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

// The widest access that divides a row: 16 bytes, 4, or 2.
inline int access_bytes(int row_bytes) { return row_bytes % 16 == 0 ? 16 : row_bytes % 4 == 0 ? 4 : 2; }

}  // namespace

cudaError_t dispatch_set_limits(int* sort_ctas) {
  const cudaError_t e = cluster_sort_limits(k_dispatch_sort<512>, 512, kMaxBins, sort_ctas);
  return e != cudaSuccess ? e : cluster_sort_limits(k_dispatch_sort<1024>, 1024, kMaxBins, sort_ctas);
}

cudaError_t launch_dispatch(const TrainDevice& d, const void* x, int row_bytes, int T, const int32_t* topk_idx,
                            int top_k, int E, int32_t* offsets, int32_t* perm, int32_t* inv, void* xs, cudaStream_t s) {
  const DispatchArgs a{topk_idx, T, top_k, E, T * top_k, offsets, perm, inv, d.status};
  const int B = access_bytes(row_bytes), nv = row_bytes / B;
  if (a.P <= kCountPairs) {
    if (B == 16) k_dispatch_count<16><<<T + 1, kThreads, 0, s>>>(a, x, nv, xs);
    else if (B == 4) k_dispatch_count<4><<<T + 1, kThreads, 0, s>>>(a, x, nv, xs);
    else k_dispatch_count<2><<<T + 1, kThreads, 0, s>>>(a, x, nv, xs);
    return cudaGetLastError();
  }
  // 512 threads a CTA have less to set up (5.3 against 6.1 us at 4160 pairs), 1024 place many pairs sooner
  // (12.2 against 13.9 us at 131072)
  const bool many = a.P > 32768;
  cudaError_t e = many ? launch_cluster_sort(d, k_dispatch_sort<1024>, 1024, a.P, E, s, a)
                       : launch_cluster_sort(d, k_dispatch_sort<512>, 512, a.P, E, s, a);
  if (e != cudaSuccess || !x) return e;
  const int q = B == 16 ? 1 : 4, nq = (nv + q - 1) / q;
  const int64_t total = (int64_t)T * nq;
  return launch_after(B == 16 ? k_dispatch_copy<16, 1> : B == 4 ? k_dispatch_copy<4, 4> : k_dispatch_copy<2, 4>,
                      blocks_of(total, kThreads), kThreads, s, x, total, nv, nq, top_k, inv, xs);
}

cudaError_t launch_combine(const TrainDevice& d, const void* ys, int dtype, int T, int H, int top_k, const int32_t* inv,
                           const float* w, void* out, cudaStream_t s) {
  const int64_t P = (int64_t)T * top_k;
  return with_dtype(dtype, [&](auto type) {
    using V = decltype(type);
    const V* y = static_cast<const V*>(ys);
    V* o = static_cast<V*>(out);
    auto launch = [&](auto n, auto columns) {
      constexpr int N = decltype(n)::value, Q = decltype(columns)::value;
      const int nv = H / N, nq = (nv + Q - 1) / Q;
      const int64_t total = (int64_t)T * nq;
      const auto kernel = w ? k_combine<V, N, Q, true> : k_combine<V, N, Q, false>;
      kernel<<<blocks_of(total, kThreads), kThreads, 0, s>>>(y, total, nv, nq, top_k, P, inv, w, o, d.status);
    };
    constexpr int N = 16 / sizeof(V);
    if (H % N == 0) launch(std::integral_constant<int, N>(), std::integral_constant<int, 1>());
    else launch(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
    return cudaGetLastError();
  });
}

cudaError_t launch_combine_backward(const TrainDevice& d, const void* dout, const void* ys, int dtype, int T, int H,
                                    int top_k, const int32_t* inv, const float* w, void* dys, float* dw,
                                    cudaStream_t s) {
  const int64_t P = (int64_t)T * top_k;
  return with_dtype(dtype, [&](auto type) {
    using V = decltype(type);
    const V *g = static_cast<const V*>(dout), *y = static_cast<const V*>(ys);
    V* o = static_cast<V*>(dys);
    auto launch = [&](auto n, auto columns, auto warps) {
      constexpr int N = decltype(n)::value, Q = decltype(columns)::value, W = decltype(warps)::value;
      k_combine_backward<V, N, Q, W><<<blocks_of(T, kThreads / 32 / W), kThreads, 0, s>>>(g, y, T, H / N, top_k, P, inv,
                                                                                          w, o, dw, d.status);
    };
    auto pick = [&](auto n, auto columns) {
      // Warps a token, so that few tokens fill the SMs: bf16 H=2560 k=8 with 1, 2, 4 or 8 takes 17.0, 10.3, 8.0,
      // 7.1 us at T=300, 24.9, 16.6, 14.0, 15.8 us at T=512, 27.2, 21.0, 23.3, 26.2 us at T=1000 and 31.6, 33.1,
      // 32.3, 34.4 us at T=1500.  Rows moved value by value keep two (172 against 142 us at T=16384 H=1001), and no
      // warp is without a piece of the row.
      const int sms = d.num_sms, pieces = H / decltype(n)::value / decltype(columns)::value;
      int W = T >= 8 * sms ? 1 : T >= 4 * sms ? 2 : T >= 5 * sms / 2 ? 4 : 8;
      if (decltype(n)::value == 1) W = std::max(W, 2);
      while (W > 1 && 32 * (W - 1) >= pieces) W /= 2;
      if (W == 1) launch(n, columns, std::integral_constant<int, 1>());
      else if (W == 2) launch(n, columns, std::integral_constant<int, 2>());
      else if (W == 4) launch(n, columns, std::integral_constant<int, 4>());
      else launch(n, columns, std::integral_constant<int, 8>());
    };
    constexpr int N = 16 / sizeof(V);
    if (H % N == 0) pick(std::integral_constant<int, N>(), std::integral_constant<int, 1>());
    else pick(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
    return cudaGetLastError();
  });
}

cudaError_t launch_route_backward(const TrainDevice& d, const float* logits, const int32_t* topk_idx,
                                  const float* topk_w, const float* dw, int T, int E, int top_k, int norm,
                                  float* dlogits, cudaStream_t s) {
  auto launch = [&](auto kernel) {
    kernel<<<blocks_of(T, kThreads / 32), kThreads, 0, s>>>(logits, topk_idx, topk_w, dw, T, E, top_k, dlogits,
                                                            d.status);
  };
  const bool wide = E % 4 == 0 && ((uintptr_t)dlogits & 15) == 0;
  if (norm) launch(wide ? k_route_backward<true, 4> : k_route_backward<true, 1>);
  else launch(wide ? k_route_backward<false, 4> : k_route_backward<false, 1>);
  return cudaGetLastError();
}

}  // namespace ftmoe
