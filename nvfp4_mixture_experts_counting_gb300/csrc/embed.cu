// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[n] = scale * table[ids[n]]
//   dtable[v] = scale * sum over the n with ids[n] = v of dout[n]   (v = padding_id: 0)
//
// The gradient sorts the tokens by id (a stable radix sort by one cluster),
// sums each run of equal ids in the order of the tokens in fp32, and writes
// every row of dtable once: no atomics, so the result does not depend on
// which CTA came first.
#include "cluster_sort.cuh"

namespace ftmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 32;     // sorted tokens that a warp sums (one per lane)
constexpr int kAhead = 8;      // rows of them in flight
constexpr int kZeroRows = 8;   // table rows that a warp fills with zeros
constexpr int kDigitBits = 10; // widest radix digit
constexpr int kSortCtas = 8;

inline int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
inline unsigned blocks_of(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

template <typename T, int N, typename Id>
__global__ void __launch_bounds__(kThreads) k_embed(const T* table, int64_t V, int nv, const Id* ids, int64_t total,
                                                    float scale, T* out, uint32_t* status) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const int64_t n = i / nv, v = i - n * nv;
  const int64_t id = ids[n];
  Pack<T, N> o;
  if (id >= 0 && id < V) {
    const Pack<T, N> r = load_pack<T, N>(table + (id * nv + v) * N);
#pragma unroll
    for (int c = 0; c < N; ++c) o.set(c, scale * r.get(c));
  } else {
    if (v == 0) set_status(status, kStatusRange);
#pragma unroll
    for (int c = 0; c < N; ++c) o.set(c, 0.f);
  }
  store_pack<T, N>(out + i * N, o);
}

// keys[final] sorted, pos[final] the tokens in that order.  A token whose id
// is the padding id or out of range gets key V, so it sorts behind all others.
template <typename Id>
__global__ void __launch_bounds__(kSortCtaThreads) k_embed_sort(const Id* ids, int64_t N, int64_t V, int64_t padding_id,
                                                                int passes, int digit, int32_t* k0, int32_t* k1,
                                                                int32_t* p0, int32_t* p1, uint32_t* status) {
  extern __shared__ int sort_smem[];
  bool bad = false;
  for (int pass = 0; pass < passes; ++pass) {
    const int32_t *src_k = pass & 1 ? k0 : k1, *src_p = pass & 1 ? p0 : p1;
    int32_t *dst_k = pass & 1 ? k1 : k0, *dst_p = pass & 1 ? p1 : p0;
    const int shift = pass * digit;
    auto full = [&](int64_t i) -> int {
      if (pass) return src_k[i];
      const int64_t id = ids[i];
      const bool in = id >= 0 && id < V;
      bad |= !in && id != padding_id;
      return in && id != padding_id ? (int)id : (int)V;
    };
    cluster_sort(
        N, 1 << digit, sort_smem, [&](int64_t i) { return (full(i) >> shift) & ((1 << digit) - 1); },
        [&](int64_t i, int, int at) {
          dst_k[at] = full(i);
          dst_p[at] = pass ? src_p[i] : (int)i;
        },
        [](int, int) {});
  }
  if (bad) set_status(status, kStatusRange);
}

struct GradArgs {
  const int32_t *keys, *pos;
  int64_t N, V;
  int nv;
  float scale;
  float* part;  // [2 * chunks][H]: a chunk's first run if it began earlier, its last if it goes on
  int accumulate;
  int64_t grad_tasks, zero_tasks;  // warps' tasks: (chunk, slice), blocks of kZeroRows rows
  int slices;
};

template <typename TT, int N>
__device__ __forceinline__ void write_row(TT* dtable, int64_t at, const float (&acc)[N], float scale, int accumulate) {
  Pack<TT, N> o;
  if (accumulate) o = load_pack<TT, N>(dtable + at);
#pragma unroll
  for (int c = 0; c < N; ++c) o.set(c, accumulate ? fmaf(scale, acc[c], o.get(c)) : scale * acc[c]);
  store_pack<TT, N>(dtable + at, o);
}

// A warp sums kChunk sorted tokens over 32 pieces of their rows.  A run that
// lies inside the chunk goes to its row; pieces of longer runs go to `part`.
// Further warps fill the rows that no token names.
template <typename T, typename TT, int N>
__global__ void __launch_bounds__(kThreads) k_embed_grad(GradArgs a, const T* dout, TT* dtable) {
  const int lane = threadIdx.x & 31;
  int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t H = (int64_t)a.nv * N;
  if (task >= a.grad_tasks) {
    task -= a.grad_tasks;
    if (task >= a.zero_tasks) return;
    // which of the rows does a token name: the first key not below the row, per lane
    const int64_t v0 = task * kZeroRows;
    bool named = true;
    if (lane < kZeroRows && v0 + lane < a.V) {
      int64_t lo = 0, hi = a.N;
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.keys[mid] < v0 + lane) lo = mid + 1;
        else hi = mid;
      }
      named = lo < a.N && a.keys[lo] == v0 + lane;
    }
    unsigned todo = __ballot_sync(0xffffffffu, !named);
    Pack<TT, N> zero;
#pragma unroll
    for (int c = 0; c < N; ++c) zero.set(c, 0.f);
    for (; todo; todo &= todo - 1) {
      TT* row = dtable + (v0 + __ffs(todo) - 1) * H;
      for (int v = lane; v < a.nv; v += 32) store_pack<TT, N>(row + (int64_t)v * N, zero);
    }
    return;
  }
  const int64_t chunk = task / a.slices, s0 = chunk * kChunk;
  const int v = (int)(task - chunk * a.slices) * 32 + lane;
  const bool on = v < a.nv;
  const int key = s0 + lane < a.N ? a.keys[s0 + lane] : (int)a.V;
  const int pos = s0 + lane < a.N ? a.pos[s0 + lane] : 0;
  const int prev = s0 > 0 ? a.keys[s0 - 1] : -1;
  const int next = s0 + kChunk < a.N ? a.keys[s0 + kChunk] : -1;
  float acc[N] = {};
  bool head = true;  // the run began at the chunk's first token
#pragma unroll 1
  for (int i0 = 0; i0 < kChunk; i0 += kAhead) {
    Pack<T, N> row[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = __shfl_sync(0xffffffffu, key, i0 + i);
      const int64_t p = __shfl_sync(0xffffffffu, pos, i0 + i);
      if (on && k < a.V) row[i] = load_pack<T, N>(dout + (p * a.nv + v) * N);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = __shfl_sync(0xffffffffu, key, i0 + i);
      const int after = __shfl_sync(0xffffffffu, key, (i0 + i + 1) & 31);
      const bool end = i0 + i == kChunk - 1;
      if (k >= a.V) return;  // padding and what lies past the last token
#pragma unroll
      for (int c = 0; c < N; ++c) acc[c] += on ? row[i].get(c) : 0.f;
      const bool goes_on = end && next == k;
      if (end || after != k) {
        if (on) {
          if (head && prev == k) {
#pragma unroll
            for (int c = 0; c < N; ++c) a.part[(2 * chunk) * H + (int64_t)v * N + c] = acc[c];
          } else if (goes_on) {
#pragma unroll
            for (int c = 0; c < N; ++c) a.part[(2 * chunk + 1) * H + (int64_t)v * N + c] = acc[c];
          } else {
            write_row<TT, N>(dtable, k * H + (int64_t)v * N, acc, a.scale, a.accumulate);
          }
        }
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] = 0.f;
        head = false;
      }
    }
  }
}

// The rows of runs that span chunks: the CTA of the chunk in which a run
// begins adds up its pieces, warp w those of the chunks w, w + 8, ... after it,
// then the warps' sums in order.
template <typename TT, int N>
__global__ void __launch_bounds__(kThreads) k_embed_join(GradArgs a, TT* dtable) {
  __shared__ float sums[kWarps][32 * N];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t chunk = (int64_t)blockIdx.x / a.slices, s0 = chunk * kChunk, H = (int64_t)a.nv * N;
  const int v = (int)((int64_t)blockIdx.x - chunk * a.slices) * 32 + lane;
  if (s0 + kChunk >= a.N) return;
  const int key = a.keys[s0 + kChunk - 1];
  if (key >= a.V || a.keys[s0 + kChunk] != key) return;                         // nothing goes on from here
  if (a.keys[s0] == key && s0 > 0 && a.keys[s0 - 1] == key) return;             // it began earlier
  // chunks after this one that the run reaches: their first key is the run's
  int64_t lo = chunk + 1, hi = (a.N + kChunk - 1) / kChunk;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (a.keys[mid * kChunk] == key) lo = mid + 1;
    else hi = mid;
  }
  const int64_t last = lo - 1;
  float acc[N] = {};
  if (v < a.nv) {
#pragma unroll 4
    for (int64_t q = chunk + warp; q <= last; q += kWarps) {
      const float* p = a.part + (2 * q + (q == chunk ? 1 : 0)) * H + (int64_t)v * N;
#pragma unroll
      for (int c = 0; c < N; ++c) acc[c] += p[c];
    }
  }
#pragma unroll
  for (int c = 0; c < N; ++c) sums[warp][c * 32 + lane] = acc[c];
  __syncthreads();
  if (warp == 0 && v < a.nv) {
#pragma unroll
    for (int c = 0; c < N; ++c) {
      acc[c] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) acc[c] += sums[w][c * 32 + lane];
    }
    write_row<TT, N>(dtable, key * H + (int64_t)v * N, acc, a.scale, a.accumulate);
  }
}

}  // namespace

EmbedWorkspace embed_workspace(int64_t N, int H) {
  EmbedWorkspace w{};
  int64_t at = 0;
  for (int i = 0; i < 2; ++i) {
    w.keys[i] = at;
    at += align256(N * 4);
    w.pos[i] = at;
    at += align256(N * 4);
  }
  w.part = at;
  w.bytes = at + (N + kChunk - 1) / kChunk * 2 * (int64_t)H * 4;
  return w;
}

cudaError_t embed_set_limits() {
  cudaError_t e = cudaFuncSetAttribute(k_embed_sort<int32_t>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       cluster_sort_smem(1 << kDigitBits));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(k_embed_sort<int64_t>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              cluster_sort_smem(1 << kDigitBits));
}

cudaError_t launch_embed(const TrainDevice& d, const void* table, int dtype, int64_t V, int H, const void* ids,
                         int id_bytes, int64_t N, float scale, void* out, cudaStream_t s) {
  return with_dtype(dtype, [&](auto type) {
    using E = decltype(type);
    auto launch = [&](auto n, auto id) {
      constexpr int W = decltype(n)::value;
      using Id = decltype(id);
      const int64_t total = N * (H / W);
      k_embed<E, W, Id><<<blocks_of(total, kThreads), kThreads, 0, s>>>(
          static_cast<const E*>(table), V, H / W, static_cast<const Id*>(ids), total, scale, static_cast<E*>(out), d.status);
    };
    auto pick = [&](auto n) {
      if (id_bytes == 8) launch(n, int64_t());
      else launch(n, int32_t());
    };
    constexpr int W = 16 / sizeof(E);
    if (H % W == 0) pick(std::integral_constant<int, W>());
    else pick(std::integral_constant<int, 1>());
    return cudaGetLastError();
  });
}

cudaError_t launch_embed_backward(const TrainDevice& d, const void* dout, int dtype, const void* ids, int id_bytes,
                                  int64_t N, int64_t V, int H, float scale, int64_t padding_id, void* dtable,
                                  int table_dtype, bool accumulate, uint8_t* ws, cudaStream_t s) {
  const EmbedWorkspace w = embed_workspace(N, H);
  int32_t* keys[2] = {reinterpret_cast<int32_t*>(ws + w.keys[0]), reinterpret_cast<int32_t*>(ws + w.keys[1])};
  int32_t* pos[2] = {reinterpret_cast<int32_t*>(ws + w.pos[0]), reinterpret_cast<int32_t*>(ws + w.pos[1])};
  int bits = 1;
  while ((V >> bits) != 0) ++bits;  // the largest key is V
  const int passes = (bits + kDigitBits - 1) / kDigitBits, digit = (bits + passes - 1) / passes;
  cudaError_t e = cudaSuccess;
  if (N > 0) {
    if (id_bytes == 8)
      e = launch_cluster_sort(k_embed_sort<int64_t>, kSortCtas, 1 << digit, s, static_cast<const int64_t*>(ids), N, V,
                              padding_id, passes, digit, keys[0], keys[1], pos[0], pos[1], d.status);
    else
      e = launch_cluster_sort(k_embed_sort<int32_t>, kSortCtas, 1 << digit, s, static_cast<const int32_t*>(ids), N, V,
                              padding_id, passes, digit, keys[0], keys[1], pos[0], pos[1], d.status);
    if (e != cudaSuccess) return e;
  }
  const int last = (passes - 1) & 1;
  const int64_t chunks = (N + kChunk - 1) / kChunk;
  GradArgs a{};
  a.keys = keys[last];
  a.pos = pos[last];
  a.N = N;
  a.V = V;
  a.scale = scale;
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.accumulate = accumulate;
  return with_dtype(dtype, [&](auto type) {
    using E = decltype(type);
    return with_dtype(table_dtype, [&](auto ttype) -> cudaError_t {
      using TT = decltype(ttype);
      if constexpr (!std::is_same<TT, float>::value && !std::is_same<TT, E>::value) {
        return cudaErrorInvalidValue;  // refused before: the table has the gradient's type or fp32
      } else {
        auto launch = [&](auto n) {
          constexpr int W = decltype(n)::value;
          a.nv = H / W;
          a.slices = (a.nv + 31) / 32;
          a.grad_tasks = chunks * a.slices;
          a.zero_tasks = accumulate ? 0 : (V + kZeroRows - 1) / kZeroRows;
          if (const int64_t tasks = a.grad_tasks + a.zero_tasks)
            k_embed_grad<E, TT, W><<<blocks_of(tasks, kWarps), kThreads, 0, s>>>(a, static_cast<const E*>(dout),
                                                                                 static_cast<TT*>(dtable));
          if (chunks > 1) k_embed_join<TT, W><<<(unsigned)(chunks * a.slices), kThreads, 0, s>>>(a, static_cast<TT*>(dtable));
        };
        constexpr int W = 16 / sizeof(E) < 16 / sizeof(TT) ? 16 / sizeof(E) : 16 / sizeof(TT);
        if (H % W == 0) launch(std::integral_constant<int, W>());
        else launch(std::integral_constant<int, 1>());
        return cudaGetLastError();
      }
    });
  });
}

}  // namespace ftmoe
