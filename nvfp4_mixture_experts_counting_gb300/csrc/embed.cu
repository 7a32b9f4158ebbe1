// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[n] = scale * table[ids[n]]
//   dtable[v] = scale * sum over the n with ids[n] = v of dout[n]   (v = padding_id: 0)
//
// The gradient sorts the tokens by id (a stable radix sort by one cluster),
// sums each run of equal ids in fp32 in a fixed order (chunks of 32 sorted
// tokens, then the chunks), and writes or adds to every row of dtable once, so
// the result does not depend on which CTA came first.
#include <algorithm>
#include <type_traits>

#include "cluster_sort.cuh"

namespace ftmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSortThreads = 512;
constexpr int kChunk = 32;     // sorted tokens that a warp sums (one per lane)
constexpr int kAhead = 8;      // rows of them in flight
constexpr int kZeroBlocks = 1024;  // blocks of table rows whose marks a CTA holds at a time
// Widest radix digit.  More bins cost each pass the exchange of more totals, and
// may save a pass.  With the gradient of H=64, at V=262144 two passes of 10 bits
// take 3 us more than three of 7 for 8191 tokens, and 58 instead of 61 us for
// 131072; at V=1000 one of 10 instead of two of 5 takes 37 instead of 44 us there,
// and for 8191 tokens as long (15 us).
constexpr int kDigitBits = 9, kManyDigitBits = 10;
constexpr int64_t kManyTokens = 65536;
// Bytes of the table for each CTA that fills, at least: it reads all ids, however
// few rows it has.  N=16384 H=2560 bf16, with and without this limit: V=4096 44
// and 54 us, V=32000 58 and 67 us; V=131072 125 us with it, 131 with 512 KB.
constexpr int64_t kFillBytes = 128 * 1024;
constexpr int kLongRun = 16;   // chunks from which a run's sum is shared by a CTA's warps

inline int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
inline unsigned blocks_of(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

// A thread takes Q pieces of a token's row, nq apart: two 16-byte loads in
// flight bring N=16384 H=2560 bf16 from 28 to 22 us (the copy rate), and rows of
// odd widths, which move value by value, take eight.
template <typename T, int N, int Q, typename Id>
__global__ void __launch_bounds__(kThreads)
    k_embed(const T* table, int64_t V, int nv, int nq, const Id* ids, int64_t total, float scale, T* out,
            uint32_t* status) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const int64_t n = quotient(i, nq);
  const int v = (int)(i - n * nq);
  const int64_t id = ids[n];
  const bool in = id >= 0 && id < V;
  if (!in && v == 0) set_status(status, kStatusRange);
  const T* row = table + (in ? id : 0) * nv * N;
  Pack<T, N> r[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) r[q] = load_pack<T, N>(row + (int64_t)min(v + q * nq, nv - 1) * N);
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (v + q * nq >= nv) break;
    Pack<T, N> o;
#pragma unroll
    for (int c = 0; c < N; ++c) o.set(c, in ? scale * r[q].get(c) : 0.f);
    store_pack<T, N>(out + (n * nv + v + q * nq) * N, o);
  }
}

// keys[final] sorted, pos[final] the tokens in that order.  A token whose id
// is the padding id or out of range gets key V, so it sorts behind all others.
template <typename Id>
__global__ void __launch_bounds__(kSortThreads)
    k_embed_sort(const Id* ids, int64_t N, int64_t V, int64_t padding_id, int passes, int digit, int32_t* k0,
                 int32_t* k1, int32_t* p0, int32_t* p1, uint32_t* status) {
  extern __shared__ int sort_smem[];
  pdl_launch_dependents();
  bool bad = false;
  for (int pass = 0; pass < passes; ++pass) {
    const int32_t *src_k = pass & 1 ? k0 : k1, *src_p = pass & 1 ? p0 : p1;
    int32_t *dst_k = pass & 1 ? k1 : k0, *dst_p = pass & 1 ? p1 : p0;
    const int shift = pass * digit;
    auto load = [&](int64_t i) {
      if (pass) return SortItem{src_k[i], src_p[i]};
      const int64_t id = ids[i];
      const bool in = id >= 0 && id < V;
      bad |= !in && id != padding_id;
      return SortItem{in && id != padding_id ? (int)id : (int)V, (int)i};
    };
    cluster_sort<kSortThreads>(
        N, 1 << digit, sort_smem, pass == passes - 1, load,
        [&](int key) { return (key >> shift) & ((1 << digit) - 1); },
        [&](int64_t, SortItem item, int at) {
          dst_k[at] = item.key;
          dst_p[at] = item.value;
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
  int64_t grad_tasks;  // (chunk, slice), a warp each
  int slices;
  // CTAs that sum, and CTAs before them that fill rows with zeros, of 2^cta_bits (or none)
  int grad_ctas, zero_first;
  int cta_bits, row_bits;
  const void* ids;
  int id_bytes;
  int64_t padding_id;
};

// Onto the table's values the sum goes as a reduction in L2, which the warp need
// not wait for (loads and stores, run by run, took 24 instead of 18 us at N=8191
// V=32000 H=64, and as long where DRAM bounds it).  A launch adds to each value
// once, so the result has one order.  Values below the smallest normal one may
// count as zero there.
template <typename TT, int N>
__device__ __forceinline__ void write_row(TT* dtable, int64_t at, const float (&acc)[N], float scale,
                                          int accumulate) {
  if constexpr (std::is_same<TT, float>::value) {
    if (accumulate) {
      float* p = dtable + at;
      if constexpr (N % 4 == 0) {
#pragma unroll
        for (int c = 0; c < N; c += 4)
          asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p + c), "f"(scale * acc[c]),
                       "f"(scale * acc[c + 1]), "f"(scale * acc[c + 2]), "f"(scale * acc[c + 3])
                       : "memory");
      } else {
#pragma unroll
        for (int c = 0; c < N; ++c) atomicAdd(p + c, scale * acc[c]);
      }
      return;
    }
  }
  Pack<TT, N> o;
#pragma unroll
  for (int c = 0; c < N; ++c) o.set(c, scale * acc[c]);
  store_pack<TT, N>(dtable + at, o);
}

// Zeros to the rows that no token names.  The CTA looks through all ids itself
// and marks the rows it meets, so it need not wait for the sort: on the SMs that
// the sort leaves free, part of a large table is written meanwhile.  Blocks of
// 2^row_bits rows go round over 2^cta_bits CTAs.
template <typename TT, int N, typename Id>
__device__ void fill_unnamed(const GradArgs& a, const Id* ids, int cta, TT* dtable) {
  __shared__ uint32_t named[kZeroBlocks];  // a word a block of this CTA
  constexpr int M = N == 1 ? 1 : 16 / sizeof(TT);  // values of one store
  const int lane = threadIdx.x & 31, nv = a.nv * (N / M);
  const int64_t blocks = (a.V + (1 << a.row_bits) - 1) >> a.row_bits;
  Pack<TT, M> zero;
#pragma unroll
  for (int c = 0; c < M; ++c) zero.set(c, 0.f);
  for (int64_t b0 = cta; b0 < blocks; b0 += (int64_t)kZeroBlocks << a.cta_bits) {
    const int mine = (int)min((int64_t)kZeroBlocks, ((blocks - b0 - 1) >> a.cta_bits) + 1);
    for (int i = threadIdx.x; i < mine; i += kThreads) named[i] = 0;
    __syncthreads();
    auto mark = [&](int64_t id) {
      const int64_t block = id >> a.row_bits;
      if (((block - cta) & ((1 << a.cta_bits) - 1)) != 0 || id == a.padding_id) return;
      const int64_t at = (block - b0) >> a.cta_bits;
      if (at >= 0 && at < mine) atomicOr(named + at, 1u << (id & ((1 << a.row_bits) - 1)));
    };
    int64_t i = threadIdx.x;
    for (; i + 7 * kThreads < a.N; i += 8 * kThreads) {
      Id id[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) id[u] = ids[i + u * kThreads];
#pragma unroll
      for (int u = 0; u < 8; ++u) mark(id[u]);
    }
    for (; i < a.N; i += kThreads) mark(ids[i]);
    __syncthreads();
    for (int j = 0; j < mine; ++j) {
      const int64_t r0 = (b0 + ((int64_t)j << a.cta_bits)) << a.row_bits;
      const int rows = (int)min((int64_t)1 << a.row_bits, a.V - r0);
      const uint32_t bits = named[j];
      TT* first = dtable + r0 * nv * M;
      if (nv >= 32) {  // a warp a row
        for (int r = threadIdx.x >> 5; r < rows; r += kWarps) {
          if (bits >> r & 1) continue;
          TT* row = first + (int64_t)r * nv * M;
#pragma unroll 4
          for (int v = lane; v < nv; v += 32) store_pack<TT, M>(row + (int64_t)v * M, zero);
        }
      } else {
        for (unsigned q = threadIdx.x; q < (unsigned)(rows * nv); q += kThreads)
          if (!(bits >> q / (unsigned)nv & 1)) store_pack<TT, M>(first + (int64_t)q * M, zero);
      }
    }
    __syncthreads();
  }
}

// A warp sums kChunk sorted tokens over a slice of their rows, kAhead rows in
// flight.  A run that lies inside the chunk goes to its row; pieces of longer
// runs go to `part`.  A lane takes Q pieces of N values of the slice, 32 pieces
// apart; rows whose bytes are no multiple of 16 move value by value (N = 1), two
// a lane.  Together with the rows of zeros it is bound by DRAM writes: N=16384
// V=131072 H=2560 bf16 118 us for 755 MB.
template <typename T, typename TT, int N, int Q>
__global__ void __launch_bounds__(kThreads, 4) k_embed_grad(GradArgs a, const T* dout, TT* dtable) {
  const int lane = threadIdx.x & 31;
  const int64_t H = (int64_t)a.nv * N;
  pdl_launch_dependents();
  // CTAs in the order in which they start: some that fill, then those that sum, then the rest that fill
  int cta = blockIdx.x;
  if (cta < a.zero_first || cta >= a.zero_first + a.grad_ctas) {
    if (cta >= a.zero_first) cta -= a.grad_ctas;
    if (a.id_bytes == 8) fill_unnamed<TT, N>(a, static_cast<const int64_t*>(a.ids), cta, dtable);
    else fill_unnamed<TT, N>(a, static_cast<const int32_t*>(a.ids), cta, dtable);
    return;
  }
  const int64_t task = (int64_t)(cta - a.zero_first) * kWarps + (threadIdx.x >> 5);
  pdl_wait();  // keys and positions are the sort's
  if (task >= a.grad_tasks) return;
  const int64_t chunk = task / a.slices, s0 = chunk * kChunk;
  const int v = (int)(task - chunk * a.slices) * 32 * Q + lane;
  const int key = s0 + lane < a.N ? a.keys[s0 + lane] : (int)a.V;
  const int pos = s0 + lane < a.N ? a.pos[s0 + lane] : 0;  // every lane has a row that may be read
  const int prev = s0 > 0 ? a.keys[s0 - 1] : -1;
  const int next = s0 + kChunk < a.N ? a.keys[s0 + kChunk] : -1;
  float acc[Q][N] = {};
  bool head = true;  // the run began at the chunk's first token
#pragma unroll 1
  for (int i0 = 0; i0 < kChunk; i0 += kAhead) {
    if (__shfl_sync(0xffffffffu, key, i0) >= a.V) return;  // padding and what lies past the last token
    Pack<T, N> row[kAhead][Q];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const T* src = dout + __shfl_sync(0xffffffffu, pos, i0 + i) * H;
#pragma unroll
      for (int q = 0; q < Q; ++q) row[i][q] = load_pack<T, N>(src + (int64_t)min(v + q * 32, a.nv - 1) * N);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = __shfl_sync(0xffffffffu, key, i0 + i);
      const int after = __shfl_sync(0xffffffffu, key, (i0 + i + 1) & 31);
      const bool end = i0 + i == kChunk - 1;
      if (k >= a.V) return;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
#pragma unroll
        for (int c = 0; c < N; ++c) acc[q][c] += row[i][q].get(c);
      }
      if (!end && after == k) continue;
      // the run ends here, or leaves the chunk
      float* part = head && prev == k  ? a.part + 2 * chunk * H
                    : end && next == k ? a.part + (2 * chunk + 1) * H
                                       : nullptr;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int64_t at = (int64_t)(v + q * 32) * N;
        if (v + q * 32 < a.nv) {
          if (part) {
#pragma unroll
            for (int c = 0; c < N; ++c) part[at + c] = acc[q][c];
          } else {
            write_row<TT, N>(dtable, k * H + at, acc[q], a.scale, a.accumulate);
          }
        }
#pragma unroll
        for (int c = 0; c < N; ++c) acc[q][c] = 0.f;
      }
      head = false;
    }
  }
}

// Sums a run's pieces over the chunks first, first + step, ... up to last:
// `from` is the chunk in which the run begins.
template <int N>
__device__ __forceinline__ void sum_pieces(const GradArgs& a, int64_t from, int64_t first, int64_t last, int64_t step,
                                           int64_t at, float (&acc)[N]) {
  const int64_t H = (int64_t)a.nv * N;
#pragma unroll 8
  for (int64_t q = first; q <= last; q += step) {
    const float* p = a.part + (2 * q + (q == from ? 1 : 0)) * H + at;
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] += p[c];
  }
}

// The rows of runs that span chunks.  A CTA takes 32 pieces of the rows and
// kWarps chunks, warp w the run that begins in chunk w and goes on: its pieces
// are added in order.  A run of over kLongRun chunks (text has tokens that make
// up much of it) is summed by all warps: warp w takes every kWarps-th chunk,
// then the warps' sums are added in order.  Latency bounds it (some 6 us).
template <typename TT, int N>
__global__ void __launch_bounds__(kThreads) k_embed_join(GradArgs a, TT* dtable, int slices) {
  __shared__ float sums[kWarps][32 * N];
  __shared__ int64_t last_of[kWarps];  // the last chunk of a long run, or -1
  __shared__ int key_of[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t group = (int64_t)blockIdx.x / slices, H = (int64_t)a.nv * N;
  const int v = (int)((int64_t)blockIdx.x - group * slices) * 32 + lane;
  const int64_t chunk = group * kWarps + warp, s0 = chunk * kChunk, at = (int64_t)v * N;
  const int64_t chunks = (a.N + kChunk - 1) / kChunk;
  pdl_wait();
  int64_t last = -1;
  int key = 0;
  if (s0 + kChunk < a.N) {
    // the run's key, the tokens around the chunk's ends, and the first keys of the next 32 chunks, at once
    key = a.keys[s0 + kChunk - 1];
    const int after = a.keys[s0 + kChunk], begin = a.keys[s0], prev = s0 > 0 ? a.keys[s0 - 1] : -1;
    int ahead = chunk + 1 + lane < chunks ? a.keys[(chunk + 1 + lane) * kChunk] : -1;
    if (key < a.V && after == key && !(begin == key && prev == key)) {
      last = chunk;
      for (;;) {
        const unsigned same = __ballot_sync(0xffffffffu, ahead == key);
        const int n = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
        last += n;
        if (n < 32) break;
        ahead = last + 1 + lane < chunks ? a.keys[(last + 1 + lane) * kChunk] : -1;
      }
    }
  }
  const bool is_long = last - chunk >= kLongRun;
  if (last >= 0 && !is_long && v < a.nv) {
    float acc[N] = {};
    sum_pieces<N>(a, chunk, chunk, last, 1, at, acc);
    write_row<TT, N>(dtable, key * H + at, acc, a.scale, a.accumulate);
  }
  if (lane == 0) {
    last_of[warp] = is_long ? last : -1;
    key_of[warp] = key;
  }
  if (!__syncthreads_or(is_long)) return;
  for (int w = 0; w < kWarps; ++w) {
    if (last_of[w] < 0) continue;
    const int64_t from = group * kWarps + w;
    float acc[N] = {};
    if (v < a.nv) sum_pieces<N>(a, from, from + warp, last_of[w], kWarps, at, acc);
#pragma unroll
    for (int c = 0; c < N; ++c) sums[warp][c * 32 + lane] = acc[c];
    __syncthreads();
    if (warp == 0 && v < a.nv) {
#pragma unroll
      for (int c = 0; c < N; ++c) {
        acc[c] = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) acc[c] += sums[q][c * 32 + lane];
      }
      write_row<TT, N>(dtable, key_of[w] * H + at, acc, a.scale, a.accumulate);
    }
    __syncthreads();
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

cudaError_t embed_set_limits(int* sort_ctas) {
  constexpr int bins = 1 << kManyDigitBits;
  const cudaError_t e = cluster_sort_limits(k_embed_sort<int32_t>, kSortThreads, bins, sort_ctas);
  return e != cudaSuccess ? e : cluster_sort_limits(k_embed_sort<int64_t>, kSortThreads, bins, sort_ctas);
}

cudaError_t launch_embed(const TrainDevice& d, const void* table, int dtype, int64_t V, int H, const void* ids,
                         int id_bytes, int64_t N, float scale, void* out, cudaStream_t s) {
  return with_dtype(dtype, [&](auto type) {
    using E = decltype(type);
    auto launch = [&](auto n, auto columns, auto id) {
      constexpr int W = decltype(n)::value, Q = decltype(columns)::value;
      using Id = decltype(id);
      const int nv = H / W, nq = (nv + Q - 1) / Q;
      const int64_t total = N * nq;
      k_embed<E, W, Q, Id><<<blocks_of(total, kThreads), kThreads, 0, s>>>(static_cast<const E*>(table), V, nv, nq,
                                                                           static_cast<const Id*>(ids), total, scale,
                                                                           static_cast<E*>(out), d.status);
    };
    auto pick = [&](auto n, auto columns) {
      if (id_bytes == 8) launch(n, columns, int64_t());
      else launch(n, columns, int32_t());
    };
    constexpr int W = 16 / sizeof(E);
    if (H % W == 0) pick(std::integral_constant<int, W>(), std::integral_constant<int, 2>());
    else pick(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
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
  const int widest = N > kManyTokens ? kManyDigitBits : kDigitBits;
  const int passes = (bits + widest - 1) / widest, digit = (bits + passes - 1) / passes;
  cudaError_t e = cudaSuccess;
  if (N > 0) {
    if (id_bytes == 8)
      e = launch_cluster_sort(d, k_embed_sort<int64_t>, kSortThreads, N, 1 << digit, s,
                              static_cast<const int64_t*>(ids), N, V, padding_id, passes, digit, keys[0], keys[1],
                              pos[0], pos[1], d.status);
    else
      e = launch_cluster_sort(d, k_embed_sort<int32_t>, kSortThreads, N, 1 << digit, s,
                              static_cast<const int32_t*>(ids), N, V, padding_id, passes, digit, keys[0], keys[1],
                              pos[0], pos[1], d.status);
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
  a.ids = ids;
  a.id_bytes = id_bytes;
  a.padding_id = padding_id;
  return with_dtype(dtype, [&](auto type) {
    using E = decltype(type);
    return with_dtype(table_dtype, [&](auto ttype) -> cudaError_t {
      using TT = decltype(ttype);
      if constexpr (!std::is_same<TT, float>::value && !std::is_same<TT, E>::value) {
        return cudaErrorInvalidValue;  // refused before: the table has the gradient's type or fp32
      } else {
        auto launch = [&](auto n, auto columns) -> cudaError_t {
          constexpr int W = decltype(n)::value, Q = decltype(columns)::value;
          a.nv = H / W;
          a.slices = (a.nv + 32 * Q - 1) / (32 * Q);
          a.grad_tasks = chunks * a.slices;
          // Many CTAs that fill, as those end at different times (16384 tokens of a table of 1.34 GB: 260 us with 512,
          // 224 with 1024, 214 with 2048, 208 with 4096), but 2^25 ids read by all of them at most; blocks of up to
          // 32 rows.
          const int64_t bytes = V * H * (int64_t)sizeof(TT);
          while (2 << a.cta_bits <= std::min<int64_t>(2048, V) && bytes >> (a.cta_bits + 1) >= kFillBytes &&
                 (N << (a.cta_bits + 1)) <= 1 << 25)
            ++a.cta_bits;
          while (a.row_bits < 5 && (V >> (a.row_bits + 1 + a.cta_bits)) > 0) ++a.row_bits;
          const int zero_ctas = accumulate ? 0 : 1 << a.cta_bits;
          a.zero_first = std::min(zero_ctas, 4 * d.num_sms);
          a.grad_ctas = (int)blocks_of(a.grad_tasks, kWarps);
          const unsigned grid = zero_ctas + a.grad_ctas;
          if (grid == 0) return cudaSuccess;
          const E* from = static_cast<const E*>(dout);
          TT* to = static_cast<TT*>(dtable);
          if (N == 0) {  // no sort before it: it starts after whatever the stream holds
            k_embed_grad<E, TT, W, Q><<<grid, kThreads, 0, s>>>(a, from, to);
            return cudaGetLastError();
          }
          const cudaError_t err = launch_after(k_embed_grad<E, TT, W, Q>, grid, kThreads, s, a, from, to);
          if (err != cudaSuccess || chunks < 2) return err;
          const int slices = (a.nv + 31) / 32;
          return launch_after(k_embed_join<TT, W>, blocks_of(chunks, kWarps) * slices, kThreads, s, a, to, slices);
        };
        constexpr int W = 16 / sizeof(E);
        if (H % W == 0) return launch(std::integral_constant<int, W>(), std::integral_constant<int, 1>());
        return launch(std::integral_constant<int, 1>(), std::integral_constant<int, 2>());
      }
    });
  });
}

}  // namespace ftmoe
