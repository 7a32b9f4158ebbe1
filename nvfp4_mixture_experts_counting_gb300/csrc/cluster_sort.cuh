// Stable counting sort of up to kMaxBins bins by one cluster of CTAs.
#pragma once

#include <cooperative_groups.h>

#include "train_common.cuh"

namespace ftmoe {

constexpr int kSortAhead = 4;  // items of a lane in flight

// Dynamic shared memory of one CTA: per-warp counts [warps][bins], the CTA's
// totals [bins], its first places [bins], and the scan's scratch.
inline int cluster_sort_smem(int threads, int bins) { return (threads / 32 * bins + 2 * bins + 64) * 4; }

struct SortItem {
  int key, value;
};

// Places the items [0, n) of the whole cluster in the order of (bin, index):
// `load(i)` gives an item, `bin(key)` its bin in [0, bins) or a negative value
// (the item has no place), `emit(i, item, place)` takes its place, or -1.
// Returns the number of items placed; first_of(bin, place) takes each bin's
// first place (cluster rank 0 only).  Each CTA takes a contiguous part of the
// items, each warp a contiguous part of those, so counting order is index
// order and the sort is stable; the counts are whole numbers, which no order
// of addition changes.  In the placing, lanes that hold one bin find one
// another by a ballot for each of the bin's bits (a warp match takes a step
// for each distinct value: 21 us against 12 us at 131072 items of 256 bins).
// The CTAs exchange their totals through distributed shared memory, which
// needs no grid-wide wait, no global scratch and no second launch.  Latency
// bounds it: loads, barriers, and the instructions themselves, which a kernel
// this short meets for the first time, so the loops are unrolled by little.
// 4160 items of 256 bins take 4.4 us with the launch, 131072 take 11.6.
// `last`: no CTA of the cluster reads what is emitted, so the closing barrier
// need not wait for those stores (some 1000 cycles).
template <int THREADS, typename Load, typename Bin, typename Emit, typename First>
__device__ int cluster_sort(int64_t n, int bins, int* smem, bool last, Load load, Bin bin, Emit emit,
                            First first_of) {
  constexpr int kSortCtaThreads = THREADS, kSortCtaWarps = THREADS / 32;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  int* count = smem;                                // [warps][bins]
  int* total = count + kSortCtaWarps * bins;        // [bins]
  int* first = total + bins;                        // [bins]
  int* scratch = first + bins;                      // [33]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bits = 32 - __clz(max(bins - 1, 1));
  const int64_t warps = (int64_t)ranks * kSortCtaWarps, per_warp = ((n + warps - 1) / warps + 31) / 32 * 32;
  const int64_t lo = min(n, ((int64_t)rank * kSortCtaWarps + warp) * per_warp), hi = min(n, lo + per_warp);
  int* mine = count + warp * bins;
  SortItem item[kSortAhead], next[kSortAhead];
  auto load_group = [&](int64_t base, SortItem (&d)[kSortAhead]) {
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u)
      if (base + u * 32 + lane < hi) d[u] = load(base + u * 32 + lane);
  };
  load_group(lo, next);
  for (int b = lane; b < bins; b += 32) mine[b] = 0;
  __syncwarp();
#pragma unroll 1
  for (int64_t base = lo; base < hi; base += 32 * kSortAhead) {
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u) item[u] = next[u];
    load_group(base + 32 * kSortAhead, next);
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u) {
      if (base + u * 32 + lane >= hi) break;
      const int k = bin(item[u].key);
      if (k >= 0) atomicAdd(mine + k, 1);
    }
  }
  const bool again = hi - lo > 32 * kSortAhead;  // else the items are at hand
  if (again) load_group(lo, next);
  __syncthreads();
  for (int b = tid; b < bins; b += kSortCtaThreads) {
    int run = 0;
#pragma unroll 1
    for (int w0 = 0; w0 < kSortCtaWarps; w0 += 8) {
      int c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = count[(w0 + w) * bins + b];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        count[(w0 + w) * bins + b] = run;
        run += c[w];
      }
    }
    total[b] = run;
  }
  cluster.sync();
  // a bin a thread: items of it before this CTA and in all CTAs, then its first
  // place by a scan over the bins.  All CTAs' totals are asked for at once, each
  // CTA from itself on: reading them in one order made every CTA wait at the same peer.
  int placed = 0;
  for (int b0 = 0; b0 < bins; b0 += kSortCtaThreads) {
    const int b = b0 + tid;
    int before = 0, all = 0;
    if (b < bins) {
      int c[kSortCtas];
#pragma unroll
      for (int i = 0; i < kSortCtas; ++i)
        c[i] = i < ranks ? *cluster.map_shared_rank(total + b, (rank + i) & (ranks - 1)) : 0;
#pragma unroll
      for (int i = 0; i < kSortCtas; ++i) {
        before += i < ranks && rank + i >= ranks ? c[i] : 0;  // the peers before this CTA come after the wrap
        all += c[i];
      }
    }
    int inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      const int w = lane < kSortCtaWarps ? scratch[lane] : 0;
      int wi = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, wi, o);
        if (lane >= o) wi += v;
      }
      if (lane < kSortCtaWarps) scratch[lane] = wi - w;
      if (lane == 31) scratch[32] = wi;
    }
    __syncthreads();
    if (b < bins) {
      const int start = placed + scratch[warp] + inc - all;
      first[b] = start + before;
      if (rank == 0) first_of(b, start);
    }
    placed += scratch[32];
    __syncthreads();
  }
  // the peers' totals have been read
  if (last) {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  }
#pragma unroll 1
  for (int64_t base = lo; base < hi; base += 32 * kSortAhead) {
    if (again) {
#pragma unroll
      for (int u = 0; u < kSortAhead; ++u) item[u] = next[u];
      load_group(base + 32 * kSortAhead, next);
    }
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u) {
      if (base + u * 32 >= hi) break;
      const bool in = base + u * 32 + lane < hi;
      const int k = in ? bin(item[u].key) : -1;
      unsigned same = __ballot_sync(0xffffffffu, k >= 0);
#pragma unroll 2
      for (int b = 0; b < bits; ++b) {
        const unsigned ones = __ballot_sync(0xffffffffu, k >> b & 1);
        same &= k >> b & 1 ? ones : ~ones;
      }
      const int ahead = __popc(same & ((1u << lane) - 1));
      int at = 0;
      if (k >= 0) at = first[k] + mine[k];
      __syncwarp();
      if (k >= 0 && ahead == 0) mine[k] += __popc(same);
      __syncwarp();
      if (in) emit(base + u * 32 + lane, item[u], k >= 0 ? at + ahead : -1);
    }
  }
  // the peers have read this CTA's totals; unless this was the last sort, the
  // cluster sees what was emitted
  __syncwarp();
  if (last) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  else cluster.sync();
  return placed;
}

struct ClusterLaunch {
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute at[1];
  ClusterLaunch(int ctas, int threads, int bins, cudaStream_t s) {
    c.gridDim = dim3(ctas);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = cluster_sort_smem(threads, bins);
    c.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
  }
};

// Shared-memory and cluster-size limits of a cluster-sort kernel; lowers *ctas
// to the portable size if the device cannot hold a cluster of kSortCtas.
template <typename... A>
cudaError_t cluster_sort_limits(void (*k)(A...), int threads, int bins, int* ctas) {
  cudaError_t e =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, cluster_sort_smem(threads, bins));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  ClusterLaunch l(kSortCtas, threads, bins, nullptr);
  int fit = 0;
  if (cudaOccupancyMaxActiveClusters(&fit, k, &l.c) != cudaSuccess || fit < 1) {
    cudaGetLastError();
    *ctas = 8;
  }
  return cudaSuccess;
}

// Launches a cluster-sort kernel of n items as one cluster: few items need no
// more than two CTAs, whose exchange is shorter.
template <typename... A, typename... B>
cudaError_t launch_cluster_sort(const TrainDevice& d, void (*k)(A...), int threads, int64_t n, int bins, cudaStream_t s,
                                B... args) {
  ClusterLaunch l(n <= 2048 ? 2 : d.sort_ctas, threads, bins, s);
  return cudaLaunchKernelEx(&l.c, k, static_cast<A>(args)...);
}

}  // namespace ftmoe
