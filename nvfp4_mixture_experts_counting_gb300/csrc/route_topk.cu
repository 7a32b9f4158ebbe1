// Routing from logits, and its gradient.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),  c_e = s_e + b_e
//   groups: the sum of a group's one or two largest c; the top_groups best
//   the top_k largest c in them, ties to the lower index
//   w_j = scale s_j / sum_i s_i, or scale s_j
//
// Experts are ranked as by fp64 arithmetic.  Where c is a monotone function of
// the logit (no bias, and groups by their largest value) the logits themselves
// are ranked, which is exact even where fp64 scores are equal (a sigmoid of 40).  Otherwise c is computed in fp32 with
// an error bound, and a token where two values that decide are closer than
// their bounds is ranked again in fp64.  How many those are is the data's: of
// fp32 N(0, 1) logits with E = 256 and biases one token in some hundreds; many of
// logits that are equal where their biases are (16-bit ones with zero biases: the
// doubt is settled by the index, but only in fp64), of softmax scores whose
// logits spread far (the bound is in proportion to the largest score), and of
// saturated sigmoids.  The times below show what that costs.
//
// A warp takes a token; lane i holds the experts i, i + 32, ...  With the
// lanes' largest values sorted, the (k+1)-th of them is below or at the (k+1)-th
// of all values, so the few values from it on hold the choice: they are
// gathered, a lane each, and each counts those before it.  (k rounds of finding
// the largest value by two reductions took twice the instructions.)
//
// The forward call is bound by issue slots, not by its bytes (2.6 us of DRAM):
// 16384 tokens of 256 experts in eight groups with biases 22 us, two thirds of
// the slots busy, some 1060 instructions a token; without biases or groups 13; 16
// tokens 5.3 us with the call, some 2.5 on the device.  With more tokens ranked in
// fp64 (top 8 of 256, no groups): bf16 N(0, 1) logits and zero biases, sigmoid 32
// us, softmax 107; fp32 logits of deviation 6 and zero biases, sigmoid 54; softmax
// with biases in steps of 0.001, deviation 4 102, 6 180; all logits and biases
// equal, sigmoid 347 (without a bias 25, as logits alone are ranked exactly),
// softmax in groups 533.  The gradient is a launch and one pass, 16384 tokens 6 us
// in a graph: each row is written after a chain of loads (index, logit) and
// shuffles, and the grid's 16 CTAs an SM are more than are resident at once.
#include <cfloat>

#include "fp8_common.cuh"

namespace ftmoe {

namespace {

constexpr int kWarps = 4;
constexpr float kEps = 5.9604645e-8f;  // 2^-24

struct RouteKernelArgs {
  const void* logits;
  int64_t ld;
  int T, E, top_k, sigmoid, norm;
  float scale;
  const float* bias;
  int n_groups, top_groups, group_best, group_size;
  uint32_t group_magic;  // ceil(2^20 / group_size): e / group_size = e * magic >> 20 for e < 2^10
  int group_lanes;       // lanes that look at a group
  int group_quads;       // each at whole quads of experts
  int by_logit;          // c's order is the logits'
  int32_t* idx;
  float* w;
  uint32_t* status;
};

__device__ __forceinline__ bool in_groups(const RouteKernelArgs& a, uint32_t groups, int e) {
  const int g = e * a.group_magic >> 20;
  return g < a.n_groups && groups >> g * a.group_lanes & 1;
}

__device__ __forceinline__ double warp_max_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float warp_max_redux(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ double smaller(double a, double b) { return a < b ? a : b; }

// The chosen groups as a mask (group g at bit g L), from the experts' values
// c[E] (-inf: not available).  L lanes take a group.  `gap`: the least chosen
// group's value less the best other one's (infinite where there is no such pair).
// `least_in`: the smallest value that counts in this lane's group.
template <typename V>
__device__ __forceinline__ uint32_t choose_groups(const RouteKernelArgs& a, const V* c, int lane, V& gap, V& least_in) {
  const int L = a.group_lanes, g = lane / L;
  const V none = -(V)INFINITY;
  V m0 = none, m1 = none;  // the two largest
  const auto take = [&](V v) {
    m1 = larger(m1, smaller(m0, v));
    m0 = larger(m0, v);
  };
  if (g < a.n_groups) {
    const int per = (a.group_size + L - 1) / L, first = lane % L * per, n = min(per, a.group_size - first);
    const V* from = c + g * a.group_size + first;
    if (sizeof(V) == 4 && a.group_quads) {
      for (int i = 0; i < n; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(from + i);
        take(v.x), take(v.y), take(v.z), take(v.w);
      }
    } else {
      for (int i = 0; i < n; ++i) take(from[i]);
    }
  }
  for (int o = L / 2; o > 0; o >>= 1) {
    const V p0 = __shfl_xor_sync(0xffffffffu, m0, o), p1 = __shfl_xor_sync(0xffffffffu, m1, o);
    m1 = larger(larger(m1, p1), smaller(m0, p0));
    m0 = larger(m0, p0);
  }
  // one available expert counts alone
  const bool two = a.group_best == 2 && m1 != none;
  const V mine = two ? m0 + m1 : m0;
  least_in = two ? m1 : m0;
  int before = 0;
  for (int o = 0; o < a.n_groups; ++o) {
    const V other = __shfl_sync(0xffffffffu, mine, o * L);
    before += other > mine || (other == mine && o < g);
  }
  const bool head = lane % L == 0 && g < a.n_groups, in = head && before < a.top_groups;
  const uint32_t mask = __ballot_sync(0xffffffffu, in);
  if (sizeof(V) == 4) {
    const V least = -(V)warp_max_redux((float)(in ? -mine : none)), best = (V)warp_max_redux((float)(head && !in ? mine : none));
    gap = best == none ? (V)INFINITY : least - best;
  }
  return mask;
}

template <typename T>
__device__ __forceinline__ float usable_logit(const T* row, int e) {
  const float l = to_f32(row[e]);
  return l < INFINITY ? l : -INFINITY;  // NaN too
}

// What an expert is ranked by, in fp64.
struct Exact {
  double m = 0, total = 1;  // the softmax's largest logit and sum
  template <typename T>
  __device__ Exact(const RouteKernelArgs& a, const T* row, int lane) {
    if (a.sigmoid) return;
    float top = -INFINITY;
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, usable_logit(row, e));
    m = warp_max_f32(top);
    double sum = 0;
    for (int e = lane; e < a.E; e += 32) sum += exp((double)usable_logit(row, e) - m);
    total = warp_sum_d(sum);
  }
  template <typename T>
  __device__ double operator()(const RouteKernelArgs& a, const T* row, int e) const {
    const float l = usable_logit(row, e), b = a.bias ? a.bias[e] : 0.f;
    const double s = a.sigmoid ? 1 / (1 + exp(-(double)l)) : exp((double)l - m) / total;
    return l == -INFINITY || !(fabsf(b) < INFINITY) ? -INFINITY : s + b;
  }
};

// The candidates of a token and its slots.
struct Chosen {
  float value[32], slot_value[33];
  int expert[32], slot_expert[33];
};

// The candidates ranked in fp64, a lane each (an SM does two fp64 operations a
// cycle: all experts would take a warp some 5 us); returns the expert of slot
// `lane`, or -1.
template <typename T>
__device__ __noinline__ int rank_again(const RouteKernelArgs& a, const T* row, Chosen& ch, int found, int lane) {
  const Exact exact(a, row, lane);
  const int e = lane < found ? ch.expert[lane] : 0;
  const double v = lane < found ? exact(a, row, e) : -INFINITY;
  int before = 0;
  for (int o = 0; o < found; ++o) {
    const double x = __shfl_sync(0xffffffffu, v, o);
    before += x > v || (x == v && o < lane);
  }
  __syncwarp();
  if (lane < found && before < a.top_k) ch.slot_expert[before] = e;
  __syncwarp();
  return lane < min(found, a.top_k) ? ch.slot_expert[lane] : -1;
}

// The groups chosen in fp64, from the experts that may be among those that
// count in their group, a lane each.
template <typename T>
__device__ __noinline__ uint32_t groups_again(const RouteKernelArgs& a, const T* row, const Chosen& ch, int found,
                                              int lane) {
  const Exact exact(a, row, lane);
  const int e = lane < found ? ch.expert[lane] : 0, mine = lane < found ? e * a.group_magic >> 20 : -1;
  const double v = lane < found ? exact(a, row, e) : -INFINITY;
  double m0 = -INFINITY, m1 = -INFINITY;  // of group `lane`
  for (int o = 0; o < found; ++o) {
    const double x = __shfl_sync(0xffffffffu, v, o);
    if (__shfl_sync(0xffffffffu, mine, o) == lane) {
      m1 = larger(m1, smaller(m0, x));
      m0 = larger(m0, x);
    }
  }
  const double score = a.group_best == 2 && m1 != -INFINITY ? m0 + m1 : m0;
  int before = 0;
  for (int o = 0; o < a.n_groups; ++o) {
    const double x = __shfl_sync(0xffffffffu, score, o);
    before += x > score || (x == score && o < lane);
  }
  const bool in = lane < a.n_groups && before < a.top_groups;
  const bool here = __shfl_sync(0xffffffffu, in, lane / a.group_lanes);
  return __ballot_sync(0xffffffffu, here && lane % a.group_lanes == 0);
}

// The whole choice in fp64, groups too.
template <typename T>
__device__ __noinline__ int route_again(const RouteKernelArgs& a, const T* row, double* c, int lane) {
  const Exact exact(a, row, lane);
  __syncwarp();
  for (int e = lane; e < a.E; e += 32) c[e] = exact(a, row, e);
  __syncwarp();
  uint32_t groups = 0xffffffffu;
  if (a.n_groups > 1) {
    double gap, least;
    groups = choose_groups(a, c, lane, gap, least);
  }
  int mine = -1;
  for (int j = 0; j < a.top_k; ++j) {
    double best = -INFINITY;
    int at = a.E;
    for (int e = lane; e < a.E; e += 32) {
      if (a.n_groups > 1 && !in_groups(a, groups, e)) continue;
      if (c[e] > best) best = c[e], at = e;
    }
    const double top = warp_max_d(best);
    if (top == -INFINITY) break;
    at = __reduce_min_sync(0xffffffffu, best == top ? at : a.E);
    if (lane == j) mine = at;
    if (at % 32 == lane) c[at] = -INFINITY;
    __syncwarp();
  }
  return mine;
}

// The larger value; NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// 1 / (1 + exp(-l)) by the approximate power of two (4 eps) and reciprocal (2 eps).
__device__ __forceinline__ float sigmoid_quick(float l) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// The warp's values, largest in lane 0 (a bitonic sort).
__device__ __forceinline__ float sort_lanes(float v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int step = size / 2; step > 0; step >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, step);
      v = ((lane & step) == 0) == ((lane & size) == 0) ? fmaxf(v, o) : fminf(v, o);
    }
  return v;
}

// VPL: experts a lane holds.  Up to 256 experts are held to 64 registers, so
// that eight CTAs fit an SM, and the grid is no larger: what a warp works out
// of the biases serves several tokens (16384 tokens in groups 25 -> 23 us).  At
// 256 that spills some (72 bytes stored, 124 loaded).
constexpr int kCtasPerSm = 8;
template <typename T, int VPL>
__global__ void __launch_bounds__(kWarps * 32, VPL <= 8 ? kCtasPerSm : VPL == 16 ? 4 : 2) k_route_topk(const __grid_constant__ RouteKernelArgs a) {
  extern __shared__ __align__(16) double shared_c[];
  __shared__ Chosen shared_chosen[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  double* exact_c = shared_c + warp * ((a.E + 1) & ~1);
  float* shared_f = reinterpret_cast<float*>(exact_c);
  Chosen& ch = shared_chosen[warp];
  pdl_wait();
  // Of this lane's experts: the bias (-inf: not available), and the bit of the group in the mask of the chosen.
  float bias[VPL], widest = 0.f;
  uint8_t group_bit[VPL];
  bool bad_bias = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    // no read-only load: the stream's previous kernel may write the biases while this one starts
    bias[i] = a.bias && e < a.E ? a.bias[e] : 0.f;
    if (fabsf(bias[i]) < INFINITY) {
      widest = fmaxf(widest, fabsf(bias[i]));
    } else {
      bad_bias |= bias[i] != -INFINITY;
      bias[i] = -INFINITY;
    }
    group_bit[i] = (uint8_t)(min(e, a.E - 1) * a.group_magic >> 20) * a.group_lanes;
  }
  widest = warp_max_redux(widest);
  if (bad_bias) set_status(a.status, kStatusRange);
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    float c[VPL];  // the logits, then what is ranked; -inf: not available
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      c[i] = e < a.E ? to_f32(row[e]) : -INFINITY;
    }
    float top = c[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = max_nan(top, c[i]);
    if (__any_sync(0xffffffffu, !(top < INFINITY))) {
      if (!(top < INFINITY)) set_status(a.status, kStatusRange);
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        c[i] = c[i] < INFINITY ? c[i] : -INFINITY;
        top = fmaxf(top, c[i]);
      }
    }
    float total = 1.f, largest = 1.f;  // the softmax's sum; the largest score
    if (!a.sigmoid && (!a.by_logit || !a.norm)) {
      top = warp_max_redux(top);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += c[i] == -INFINITY ? 0.f : expf(c[i] - top);
      total = warp_sum_f32(sum);
      largest = 1.f / total;
    }
    float bound = 0.f;
    if (!a.by_logit) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float v = (a.sigmoid ? sigmoid_quick(c[i]) : expf(c[i] - top) * largest) + bias[i];
        c[i] = c[i] == -INFINITY ? -INFINITY : v;
      }
      // |error of s| <= 5 eps for the sigmoid: exp's 4 eps and its argument's 2 |l| eps count by s (1 - s), 1.5 in
      // all, then the sum's and the reciprocal's.  For the softmax (VPL + 18) eps of the largest s, from the
      // exponents (|l - top| eps, at most ln E in the mean of the sum), exp (2 eps), a lane's sum, the joins (5) and
      // the two products.  The bias adds eps |c|, |c| <= the largest s and bias.  Two values differ for sure beyond
      // the sum of their bounds; half is added.
      bound = 1.5f * kEps * (2.f * (a.sigmoid ? 5.f : (VPL + 18.f) * largest) + 2.f * (largest + widest));
    }
    // experts that `in` takes, in order, into ch; their number (32 are kept)
    const auto gather = [&](auto in) {
      int found = 0;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const bool yes = in(i) && c[i] != -INFINITY;
        const uint32_t mask = __ballot_sync(0xffffffffu, yes);
        const int at = found + __popc(mask & ((1u << lane) - 1));
        if (yes && at < 32) {
          ch.value[at] = c[i];
          ch.expert[at] = lane + 32 * i;
        }
        found += __popc(mask);
      }
      __syncwarp();
      return found;
    };
    bool again = false, all_again = false;  // is the order in doubt; can only all experts in fp64 settle it
    if (a.n_groups > 1) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < a.E) shared_f[lane + 32 * i] = c[i];
      __syncwarp();
      float gap, least;
      uint32_t groups = choose_groups(a, shared_f, lane, gap, least);
      if (!a.by_logit && gap <= 3.f * bound) {  // of sums of two values, which are rounded too
        const int found =
            gather([&](int i) { return c[i] >= __shfl_sync(0xffffffffu, least, group_bit[i]) - bound; });
        if (found <= 32)
          groups = groups_again(a, row, ch, found, lane);
        else
          all_again = true;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        c[i] = groups >> group_bit[i] & 1 ? c[i] : -INFINITY;
    }
    float most = c[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) most = fmaxf(most, c[i]);
    // from the (k+1)-th on, and those that may be its equals (bound is 0 where logits are ranked)
    const float from =
        a.top_k < 32 ? __shfl_sync(0xffffffffu, sort_lanes(most, lane), a.top_k & 31) - bound : -INFINITY;
    const int found = gather([&](int i) { return c[i] >= from; });
    int mine = -1;  // slot j's expert stays with lane j
    if (found <= 32) {
      const float v = lane < found ? ch.value[lane] : -INFINITY;
      int before = 0;
#pragma unroll 4
      for (int o = 0; o < found; ++o) {
        const float x = __shfl_sync(0xffffffffu, v, o);
        before += x > v || (x == v && o < lane);
      }
      if (lane < found && before <= a.top_k) {
        ch.slot_value[before] = v;
        ch.slot_expert[before] = ch.expert[lane];
      }
      __syncwarp();
      if (lane < min(found, a.top_k)) mine = ch.slot_expert[lane];
      // neighbours up to the first one left out
      if (!a.by_logit)
        again |= __any_sync(0xffffffffu, lane < a.top_k && lane + 1 < found &&
                                             ch.slot_value[lane] - ch.slot_value[lane + 1] <= bound);
    } else {
      // many equal values, or many of the largest in few lanes: the largest again and again
      float last = 0.f;
      for (int j = 0; j < a.top_k + !a.by_logit; ++j) {
        float best = -INFINITY;
        int at = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (c[i] > best) best = c[i], at = i;
        const float high = warp_max_redux(best);
        if (high == -INFINITY) break;
        if (!a.by_logit && j > 0) again |= last - high <= bound;
        last = high;
        const int e = __reduce_min_sync(0xffffffffu, best == high ? lane + 32 * at : 1 << 20);
        if (lane == j) mine = e;
        if ((e & 31) == lane) {
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            if (i == e / 32) c[i] = -INFINITY;
        }
      }
    }
    if (all_again || (again && found > 32))
      mine = route_again(a, row, exact_c, lane);
    else if (again)
      mine = rank_again(a, row, ch, found, lane);
    if (lane >= a.top_k) mine = -1;
    // weights relative to the largest chosen score, so that scores below fp32's range keep their ratios
    float s = 0.f;
    const float z = mine >= 0 ? usable_logit(row, mine) : -INFINITY;
    if (a.norm) {
      const float n = a.sigmoid ? fminf(z, 0.f) : z, high = warp_max_redux(n);
      if (mine >= 0) s = a.sigmoid ? expf(n - high) / (1.f + expf(-fabsf(z))) : expf(n - high);
      const float sum = warp_sum_f32(s);
      s = sum > 0.f ? s * a.scale / sum : 0.f;
    } else if (mine >= 0) {
      s = a.scale * (a.sigmoid ? sigmoid(z) : expf(z - top) * largest);
    }
    if (lane < a.top_k) {
      a.idx[t * a.top_k + lane] = mine;
      a.w[t * a.top_k + lane] = s;
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------- gradient

// With u = dw and D = sum_j w_j u_j, for the expert of slot j
//   softmax, norm: w_j (u_j - D / scale)   else: p_e (scale u_j - D), and -p_e D for every other expert
//   sigmoid, norm: w_j (1 - s_j) (u_j - D / scale)   else: w_j (1 - s_j) u_j
// Slots with the same expert add up.  A warp takes a token: it writes the row
// of zeros (or of -p_e D) and then the chosen places.
template <typename T, int V>
__global__ void __launch_bounds__(kWarps * 32) k_route_topk_backward(const __grid_constant__ RouteKernelArgs a,
                                                                     const float* dw, T* dlogits, int64_t ld_d) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  for (int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; t < a.T; t += (int64_t)gridDim.x * kWarps) {
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    T* out = dlogits + t * ld_d;
    int e = -1;
    float w = 0.f, u = 0.f, z = 0.f;
    if (lane < a.top_k) {
      e = a.idx[t * a.top_k + lane];
      if (e < -1 || e >= a.E) {
        set_status(a.status, kStatusRange);
        e = -1;
      }
      if (e >= 0) {
        w = a.w[t * a.top_k + lane];
        u = dw[t * a.top_k + lane];
        if (a.sigmoid || !a.norm) z = usable_logit(row, e);
      }
    }
    const float D = warp_sum_f32(w * u);
    float g;
    if (a.sigmoid)
      g = w * (a.norm ? u - D / a.scale : u) / (1.f + expf(z));
    else
      g = a.norm ? w * (u - D / a.scale) : a.scale * u;
    if (e < 0) g = 0.f;
    float sum = 0.f;  // over the slots of this expert
    for (int j = 0; j < a.top_k; ++j) {
      const int o = __shfl_sync(0xffffffffu, e, j);
      const float x = __shfl_sync(0xffffffffu, g, j);
      if (o == e) sum += x;
    }
    if (!a.sigmoid && !a.norm) {
      float top = -INFINITY, part = 0.f;
      for (int i = lane; i < a.E; i += 32) top = fmaxf(top, usable_logit(row, i));
      top = warp_max_f32(top);
      for (int i = lane; i < a.E; i += 32) {
        const float l = usable_logit(row, i);
        part += l == -INFINITY ? 0.f : expf(l - top);
      }
      const float total = warp_sum_f32(part), inv = total > 0.f ? 1.f / total : 0.f;
      const float p = z == -INFINITY ? 0.f : expf(z - top) * inv;
      for (int i = lane; i < a.E; i += 32) {
        const float l = usable_logit(row, i);
        out[i] = from_f32<T>(l == -INFINITY ? 0.f : expf(l - top) * inv * -D);
      }
      sum = p * (sum - D);
    } else {
      Pack<T, V> zero;
#pragma unroll
      for (int i = 0; i < V; ++i) zero.set(i, 0.f);
      __syncwarp();  // logits may be dlogits: the chosen ones are read
      for (int i = lane * V; i < a.E; i += 32 * V) store_pack<T, V>(out + i, zero);
    }
    __syncwarp();
    if (e >= 0) out[e] = from_f32<T>(sum);
  }
}

RouteKernelArgs kernel_args(const TrainDevice& d, const ftmoe_route_args& r) {
  RouteKernelArgs a{};
  a.logits = r.logits;
  a.ld = r.ld;
  a.T = r.T;
  a.E = r.E;
  a.top_k = r.top_k;
  a.sigmoid = r.score == FTMOE_SCORE_SIGMOID;
  a.norm = r.norm_topk_prob;
  a.scale = r.scale;
  a.bias = r.bias;
  a.n_groups = r.n_groups;
  a.top_groups = r.top_groups;
  a.group_best = r.group_best;
  a.group_size = r.E / r.n_groups;
  a.group_magic = (uint32_t)(((1 << 20) + a.group_size - 1) / a.group_size);
  a.group_lanes = 32;
  while (a.group_lanes * a.n_groups > 32) a.group_lanes >>= 1;
  a.group_quads = a.group_size % (4 * a.group_lanes) == 0;
  a.by_logit = !r.bias && (r.n_groups == 1 || r.group_best == 1);
  a.idx = r.topk_idx;
  a.w = r.topk_w;
  a.status = d.status;
  return a;
}

unsigned route_grid(const TrainDevice& d, int T, int ctas_per_sm) {
  const int need = (T - 1) / kWarps + 1, most = d.num_sms * ctas_per_sm;
  return (unsigned)(need < most ? need : most);
}

}  // namespace

cudaError_t launch_route_topk(const TrainDevice& d, const ftmoe_route_args& r, cudaStream_t s) {
  const RouteKernelArgs a = kernel_args(d, r);
  return with_dtype(r.dtype, [&](auto zero) {
    using T = decltype(zero);
    const int per = (r.E + 31) / 32;
    auto* k = per <= 1 ? k_route_topk<T, 1> : per <= 2 ? k_route_topk<T, 2> : per <= 4 ? k_route_topk<T, 4>
              : per <= 8 ? k_route_topk<T, 8> : per <= 16 ? k_route_topk<T, 16> : k_route_topk<T, 32>;
    // 32 KB at E = 1024: within what a kernel has without asking
    return launch_after_smem(k, route_grid(d, r.T, kCtasPerSm), kWarps * 32, kWarps * ((r.E + 1) & ~1) * sizeof(double), s, a);
  });
}

cudaError_t launch_route_topk_backward(const TrainDevice& d, const ftmoe_route_args& r, const float* dw, void* dlogits,
                                       int64_t ld_d, cudaStream_t s) {
  const RouteKernelArgs a = kernel_args(d, r);
  return with_dtype(r.dtype, [&](auto zero) {
    using T = decltype(zero);
    constexpr int V = 16 / sizeof(T);
    const bool wide = r.E % V == 0 && ld_d % V == 0 && ((uintptr_t)dlogits & 15) == 0;
    return launch_after(wide ? k_route_topk_backward<T, V> : k_route_topk_backward<T, 1>, route_grid(d, r.T, 16),
                        kWarps * 32, s, a, dw, static_cast<T*>(dlogits), ld_d);
  });
}

}  // namespace ftmoe
