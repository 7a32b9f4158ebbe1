// Stable counting sort of up to kMaxBins bins by one cluster of CTAs.
#pragma once

#include <cooperative_groups.h>

#include "train_common.cuh"

namespace ftmoe {

constexpr int kSortCtaThreads = 1024;
constexpr int kSortCtaWarps = kSortCtaThreads / 32;

// Dynamic shared memory of one CTA: per-warp counts [warps][bins], the CTA's
// totals [bins], its first places [bins], and the scan's scratch.
inline int cluster_sort_smem(int bins) { return (kSortCtaWarps * bins + 2 * bins + 64) * 4; }

// Places the items [0, n) of the whole cluster in the order of (key, index):
// `key(i)` gives an item's bin in [0, bins) or a negative value (the item has
// no place), `emit(i, key, place)` takes its place, or -1.  Returns the number of
// items placed; first_of(bin, place) takes each bin's first place (cluster
// rank 0 only).  Each CTA takes a contiguous part of the items, each warp a
// contiguous part of those, so counting order is index order and the sort is
// stable without an atomic: lanes that hold one key find one another with a
// warp match, and one of them adds their number to the warp's own count.
// The CTAs exchange their totals through distributed shared memory, which
// needs no grid-wide wait, no global scratch and no second launch.
template <typename Key, typename Emit, typename First>
__device__ int cluster_sort(int64_t n, int bins, int* smem, Key key, Emit emit, First first_of) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  int* count = smem;                                // [warps][bins]
  int* total = count + kSortCtaWarps * bins;        // [bins]
  int* first = total + bins;                        // [bins]
  int* scratch = first + bins;                      // [33]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t per_warp = ((n + (int64_t)ranks * kSortCtaWarps - 1) / ((int64_t)ranks * kSortCtaWarps) + 31) / 32 * 32;
  const int64_t lo = min(n, ((int64_t)rank * kSortCtaWarps + warp) * per_warp), hi = min(n, lo + per_warp);
  int* mine = count + warp * bins;
  for (int b = lane; b < bins; b += 32) mine[b] = 0;
  __syncwarp();
  for (int64_t i = lo; i < hi; i += 32) {
    const int k = i + lane < hi ? key(i + lane) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, k);
    if (k >= 0 && (same & ((1u << lane) - 1)) == 0) mine[k] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int b = tid; b < bins; b += kSortCtaThreads) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < kSortCtaWarps; ++w) {
      const int c = count[w * bins + b];
      count[w * bins + b] = run;
      run += c;
    }
    total[b] = run;
  }
  cluster.sync();
  // one bin a thread: items of it before this CTA, and in all CTAs
  int before = 0, all = 0;
  if (tid < bins) {
    for (int r = 0; r < ranks; ++r) {
      const int c = *cluster.map_shared_rank(total + tid, r);
      before += r < rank ? c : 0;
      all += c;
    }
  }
  int inc = all;  // inclusive scan over the bins
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = scratch[lane];
    int wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += v;
    }
    scratch[lane] = wi - w;
    if (lane == 31) scratch[32] = wi;
  }
  __syncthreads();
  const int placed = scratch[32];
  if (tid < bins) {
    const int start = scratch[warp] + inc - all;
    first[tid] = start + before;
    if (rank == 0) first_of(tid, start);
  }
  __syncthreads();
  for (int64_t i = lo; i < hi; i += 32) {
    const bool in = i + lane < hi;
    const int k = in ? key(i + lane) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, k);
    const int ahead = __popc(same & ((1u << lane) - 1));
    int base = 0;
    if (k >= 0) base = first[k] + mine[k];
    __syncwarp();
    if (k >= 0 && ahead == 0) mine[k] += __popc(same);
    __syncwarp();
    if (in) emit(i + lane, k, k >= 0 ? base + ahead : -1);
  }
  cluster.sync();  // the peers have read this CTA's totals; what was emitted is seen by the whole cluster
  return placed;
}

// Launches a cluster-sort kernel as one cluster of `ctas` CTAs.
template <typename... A, typename... B>
cudaError_t launch_cluster_sort(void (*k)(A...), int ctas, int bins, cudaStream_t s, B... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(ctas);
  c.blockDim = dim3(kSortCtaThreads);
  c.dynamicSmemBytes = cluster_sort_smem(bins);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, args...);
}

}  // namespace ftmoe
