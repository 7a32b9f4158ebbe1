// One AdamW step over many tensors, with states in 32 bits or in 8.
//
// With g' = grad_scale * g and t the step's number from 1:
//   m <- b1 m + (1 - b1) g',  v <- b2 v + (1 - b2) g'^2
//   p <- p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32.  m and v are computed with each operation rounded on its own (no
// contraction), so that the 8-bit codes below are those of the formula, bit for bit.
//
// 8 bits: m and the root u = sqrt(v) are E4M3 codes with one fp32 scale for
// each 256 values of the tensor, scale = amax * fl(1/448), code = E4M3(x *
// (448 * fl(1/amax))).  The root and not v is held: its codes then span 2^17
// in u, 2^34 in v, and the update divides by u.  A root that is not zero never
// rounds to zero, which would make the next step's divisor eps alone.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "train_common.cuh"

namespace ftmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                  // values a thread updates
constexpr int kTile = kThreads * kPer;   // a CTA's values, 32-bit states
constexpr int kMaxTileBlocks = 32;       // a CTA's 256-value blocks, 8-bit states
// Tensors of one launch: the descriptors travel as kernel parameters, and
// 29 KB of them cost some 3 us of the launch, so short lists have a kernel of their own.
constexpr int kFewTensors = 24, kMaxTensors = 360;
constexpr float kTiny = 1e-30f;          // blocks below it are held as zeros

struct Tensor {
  void* p;
  const void* g;
  float* master;
  void *m, *v;
  float *m_scale, *v_scale;
  int64_t n;
  uint32_t tile0;  // the tensor's first tile in the launch
  float decay;     // 1 - lr wd
  uint32_t aligned;  // 8-bit states: every array starts where 8 of its values move in whole accesses
};

struct Common {
  float b1, ob1, b2, ob2, root_scale, eps, lr;
  const float* grad_scale;
  int count;
  int tile_blocks;  // 8-bit states: a tile's blocks
};
template <int CAP>
struct Launch : Common {
  Tensor t[CAP];
};
static_assert(sizeof(Launch<kMaxTensors>) <= 32764, "kernel parameters");

// kPer consecutive values from `i` on; past n they are zeros.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t i, int64_t n, float (&f)[kPer]) {
  constexpr int N = 16 / sizeof(T) < kPer ? 16 / sizeof(T) : kPer;
  if (i + kPer <= n && ((uintptr_t)(p + i) & (sizeof(T) * N - 1)) == 0) {
#pragma unroll
    for (int c = 0; c < kPer; c += N) {
      const Pack<T, N> r = load_pack<T, N>(p + i + c);
#pragma unroll
      for (int e = 0; e < N; ++e) f[c + e] = r.get(e);
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < kPer; ++c) f[c] = i + c < n ? to_f32(p[i + c]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t i, int64_t n, const float (&f)[kPer]) {
  constexpr int N = 16 / sizeof(T) < kPer ? 16 / sizeof(T) : kPer;
  if (i + kPer <= n && ((uintptr_t)(p + i) & (sizeof(T) * N - 1)) == 0) {
#pragma unroll
    for (int c = 0; c < kPer; c += N) {
      Pack<T, N> r;
#pragma unroll
      for (int e = 0; e < N; ++e) r.set(e, f[c + e]);
      store_pack<T, N>(p + i + c, r);
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < kPer; ++c)
    if (i + c < n) p[i + c] = from_f32<T>(f[c]);
}

// The launch's tensor that tile `tile` belongs to: the last that starts at or before it.
template <int CAP>
__device__ __forceinline__ const Tensor& tensor_of(const Launch<CAP>& a, uint32_t tile) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].tile0 <= tile) lo = mid;
    else hi = mid - 1;
  }
  return a.t[lo];
}

// States in 32 bits: a thread's kPer values are loaded, updated and stored.
// The step moves 28 bytes a value (bf16 weight and gradient, fp32 master and
// states) for some 40 instructions, so memory bounds it: 267 M values take
// 1062 us, 7.05 TB/s.
template <typename PT, typename GT, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ Launch<CAP> a) {
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  if (!isfinite(gs)) return;  // an overflowed step is skipped
  const Tensor& t = tensor_of(a, blockIdx.x);
  const int64_t i = (int64_t)(blockIdx.x - t.tile0) * kTile + threadIdx.x * kPer, n = t.n;
  if (i >= n) return;
  float p[kPer], g[kPer], m[kPer], v[kPer];
  load8(static_cast<const GT*>(t.g), i, n, g);
  if (MASTER) load8(static_cast<const float*>(t.master), i, n, p);
  else load8(static_cast<const PT*>(t.p), i, n, p);
  load8(static_cast<const float*>(t.m), i, n, m);
  load8(static_cast<const float*>(t.v), i, n, v);
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const float gc = __fmul_rn(g[c], gs);
    m[c] = __fadd_rn(__fmul_rn(m[c], a.b1), __fmul_rn(gc, a.ob1));
    v[c] = __fadd_rn(__fmul_rn(v[c], a.b2), __fmul_rn(__fmul_rn(gc, gc), a.ob2));
    const float update = __fdiv_rn(m[c], fmaf(__fsqrt_rn(v[c]), a.root_scale, a.eps));
    p[c] = fmaf(-update, a.lr, p[c] * t.decay);
  }
  store8(static_cast<PT*>(t.p), i, n, p);
  if (MASTER) store8(t.master, i, n, p);
  store8(static_cast<float*>(t.m), i, n, m);
  store8(static_cast<float*>(t.v), i, n, v);
}

// A lane's 8 values of one block, as they lie in memory.
template <typename PT, typename GT, bool MASTER>
struct Block8 {
  using WT = typename std::conditional<MASTER, float, PT>::type;  // what is updated
  Pack<GT, 16 / sizeof(GT)> g[sizeof(GT) / 2];
  Pack<WT, 16 / sizeof(WT)> p[sizeof(WT) / 2];
  uint2 m, u;
  float m_scale, u_scale;
};

// Values past the tensor's end read as zero codes and zero gradients, and are not written.
template <bool FULL, typename T>
__device__ __forceinline__ void load_values(const T* src, int64_t i, int64_t n,
                                            Pack<T, 16 / sizeof(T)> (&d)[sizeof(T) / 2]) {
  constexpr int N = 16 / sizeof(T);
#pragma unroll
  for (int q = 0; q < (int)sizeof(T) / 2; ++q) {
    if constexpr (FULL) {
      d[q] = load_pack<T, N>(src + i + q * N);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) d[q].v[e] = i + q * N + e < n ? src[i + q * N + e] : from_f32<T>(0.f);
    }
  }
}
template <bool FULL>
__device__ __forceinline__ uint2 load_codes(const uint8_t* src, int64_t i, int64_t n) {
  if constexpr (FULL) {
    return *reinterpret_cast<const uint2*>(src + i);
  } else {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (i + c < n) w[c / 4] |= (uint32_t)src[i + c] << (c % 4 * 8);
    return make_uint2(w[0], w[1]);
  }
}
template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t* dst, int64_t i, int64_t n, uint2 v) {
  if constexpr (FULL) {
    *reinterpret_cast<uint2*>(dst + i) = v;
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (i + c < n) dst[i + c] = (uint8_t)((c < 4 ? v.x : v.y) >> (c % 4 * 8));
  }
}

template <bool FULL, typename PT, typename GT, bool MASTER>
__device__ __forceinline__ Block8<PT, GT, MASTER> load_block(const Tensor& t, int64_t block, int lane) {
  Block8<PT, GT, MASTER> b;
  using WT = typename Block8<PT, GT, MASTER>::WT;
  const int64_t i = block * 256 + lane * kPer;
  load_values<FULL>(static_cast<const GT*>(t.g), i, t.n, b.g);
  load_values<FULL>(MASTER ? reinterpret_cast<const WT*>(t.master) : static_cast<const WT*>(t.p), i, t.n, b.p);
  b.m = load_codes<FULL>(static_cast<const uint8_t*>(t.m), i, t.n);
  b.u = load_codes<FULL>(static_cast<const uint8_t*>(t.v), i, t.n);
  b.m_scale = t.m_scale[block];
  b.u_scale = t.v_scale[block];
  return b;
}

// Two E4M3 codes as fp32 values, and the codes of two values.
__device__ __forceinline__ uint64_t decode2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
  return pack2(f.x, f.y);
}
__device__ __forceinline__ uint32_t encode2(uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t half_of(uint2 w, int e) { return (e < 2 ? w.x : w.y) >> (e % 2 * 16); }

// A sum of two products, each rounded on its own: the compiler fuses a packed
// sum with the packed product before it, so the sum is taken value by value.
__device__ __forceinline__ uint64_t add_apart(uint64_t a, uint64_t b) {
  float a0, a1, b0, b1;
  unpack2(a, a0, a1);
  unpack2(b, b0, b1);
  return pack2(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}

// One block of 256 values by a warp.  Memory moves 10 bytes a value (bf16
// weight, gradient and two codes), so the instructions count: pairs of values
// share one where the hardware has it, the two scales' reciprocals are taken by
// two lanes at once, and the quotient, which only the weight sees, is a product
// with an approximate reciprocal (2 ulp of the update): 87 instructions a value
// became 56.
template <bool FULL, typename PT, typename GT, bool MASTER, int CAP>
__device__ __forceinline__ void step_block(const Launch<CAP>& a, const Tensor& t, int64_t block, int lane, float gs,
                                           const Block8<PT, GT, MASTER>& b) {
  using WT = typename Block8<PT, GT, MASTER>::WT;
  constexpr int GN = 16 / sizeof(GT), WN = 16 / sizeof(WT), PN = 16 / sizeof(PT);
  const int64_t i = block * 256 + lane * kPer;
  uint64_t m[kPer / 2], u[kPer / 2];
  Pack<WT, WN> w[sizeof(WT) / 2];
  Pack<PT, PN> out[sizeof(PT) / 2];
  float top_m = 0.f, top_u = 0.f, low_u = INFINITY;
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) {
    const uint64_t g = mul2(pair_of(b.g[2 * e / GN], e % (GN / 2)), pack2(gs, gs));
    m[e] = mul2(decode2(half_of(b.m, e)), pack2(b.m_scale, b.m_scale));
    m[e] = add_apart(mul2(m[e], pack2(a.b1, a.b1)), mul2(g, pack2(a.ob1, a.ob1)));
    const uint64_t old = mul2(decode2(half_of(b.u, e)), pack2(b.u_scale, b.u_scale));
    const uint64_t v = add_apart(mul2(mul2(old, old), pack2(a.b2, a.b2)), mul2(mul2(g, g), pack2(a.ob2, a.ob2)));
    float v0, v1, m0, m1, d0, d1;
    unpack2(v, v0, v1);
    v0 = __fsqrt_rn(v0);
    v1 = __fsqrt_rn(v1);
    u[e] = pack2(v0, v1);
    unpack2(m[e], m0, m1);
    unpack2(fma2(u[e], pack2(a.root_scale, a.root_scale), pack2(a.eps, a.eps)), d0, d1);
    const uint64_t update = pack2(__fdividef(m0, d0), __fdividef(m1, d1));
    const uint64_t kept = mul2(pair_of(b.p[2 * e / WN], e % (WN / 2)), pack2(t.decay, t.decay));
    const uint64_t p = fma2(update, pack2(-a.lr, -a.lr), kept);
    set_pair(w[2 * e / WN], e % (WN / 2), p);
    if (MASTER) set_pair(out[2 * e / PN], e % (PN / 2), p);
    top_m = fmaxf(top_m, fmaxf(fabsf(m0), fabsf(m1)));
    top_u = fmaxf(top_u, fmaxf(v0, v1));
    low_u = fminf(low_u, fminf(v0, v1));
  }
  // the two largest (bits of values that are not negative order as integers do), a lane each for the scales
  top_m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_m)));
  top_u = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_u)));
  const float top = lane & 1 ? top_u : top_m;
  const float r = top < kTiny ? 0.f : __fmul_rn(__frcp_rn(top), 448.f);
  if (lane < 2) (lane ? t.v_scale : t.m_scale)[block] = top < kTiny ? 0.f : __fmul_rn(top, 1.f / 448.f);
  const float rm = __shfl_sync(0xffffffffu, r, 0), ru = __shfl_sync(0xffffffffu, r, 1);
  uint32_t cm[kPer / 2], cu[kPer / 2];
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) {
    cm[e] = encode2(mul2(m[e], pack2(rm, rm)));
    cu[e] = encode2(mul2(u[e], pack2(ru, ru)));
  }
  if (low_u * ru < 0x1p-9f && ru > 0.f) {  // a root above zero keeps the smallest code
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) {
      float v0, v1;
      unpack2(u[e], v0, v1);
      if ((cu[e] & 0xff) == 0 && v0 > 0.f) cu[e] |= 1;
      if ((cu[e] & 0xff00) == 0 && v1 > 0.f) cu[e] |= 0x100;
    }
  }
  store_codes<FULL>(static_cast<uint8_t*>(t.m), i, t.n, make_uint2(cm[0] | cm[1] << 16, cm[2] | cm[3] << 16));
  store_codes<FULL>(static_cast<uint8_t*>(t.v), i, t.n, make_uint2(cu[0] | cu[1] << 16, cu[2] | cu[3] << 16));
  WT* dst = MASTER ? reinterpret_cast<WT*>(t.master) : static_cast<WT*>(t.p);
#pragma unroll
  for (int q = 0; q < (int)sizeof(WT) / 2; ++q) {
    if constexpr (FULL) {
      store_pack<WT, WN>(dst + i + q * WN, w[q]);
    } else {
#pragma unroll
      for (int e = 0; e < WN; ++e)
        if (i + q * WN + e < t.n) dst[i + q * WN + e] = w[q].v[e];
    }
  }
  if (MASTER) {
    PT* p = static_cast<PT*>(t.p);
#pragma unroll
    for (int q = 0; q < (int)sizeof(PT) / 2; ++q) {
      if constexpr (FULL) {
        store_pack<PT, PN>(p + i + q * PN, out[q]);
      } else {
#pragma unroll
        for (int e = 0; e < PN; ++e)
          if (i + q * PN + e < t.n) p[i + q * PN + e] = out[q].v[e];
      }
    }
  }
}

// States in 8 bits: a CTA is one warp, which goes through its tile's blocks
// with the next one's values on their way while it updates one.  With 32 such CTAs an
// SM and 32 blocks each, 267 M values take 408 us (97% of the copy rate); two warps
// a CTA take 425 us, four 472 us and eight 565 us, as a CTA then holds its place
// until its last warp is done.  A tensor with an array off its alignment moves
// value by value (64 M values: 215 us instead of 117).
template <typename PT, typename GT, bool MASTER, int CAP>
__global__ void __launch_bounds__(32, 32) k_adamw_8bit(const __grid_constant__ Launch<CAP> a) {
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  if (!isfinite(gs)) return;  // an overflowed step is skipped
  const Tensor& t = tensor_of(a, blockIdx.x);
  const int lane = threadIdx.x;
  int64_t block = (int64_t)(blockIdx.x - t.tile0) * a.tile_blocks;
  const int64_t tile_end = block + a.tile_blocks;
  const int64_t whole = min(tile_end, t.aligned ? t.n / 256 : 0), end = min(tile_end, (t.n + 255) / 256);
  if (block < whole) {
    auto b = load_block<true, PT, GT, MASTER>(t, block, lane);
    for (; block + 1 < whole; ++block) {
      const auto next = load_block<true, PT, GT, MASTER>(t, block + 1, lane);
      step_block<true, PT, GT, MASTER>(a, t, block, lane, gs, b);
      b = next;
    }
    step_block<true, PT, GT, MASTER>(a, t, block, lane, gs, b);
    ++block;
  }
  for (; block < end; ++block)
    step_block<false, PT, GT, MASTER>(a, t, block, lane, gs, load_block<false, PT, GT, MASTER>(t, block, lane));
}

template <typename PT, typename GT, bool MASTER, int CAP>
void launch_size(bool eight, uint32_t tiles, const Launch<CAP>& l, cudaStream_t s) {
  if (eight) k_adamw_8bit<PT, GT, MASTER><<<tiles, 32, 0, s>>>(l);
  else k_adamw<PT, GT, MASTER><<<tiles, kThreads, 0, s>>>(l);
}

template <typename PT, typename GT, bool MASTER>
void launch_kind(bool eight, uint32_t tiles, const Launch<kMaxTensors>& l, cudaStream_t s) {
  if (l.count <= kFewTensors) {
    Launch<kFewTensors> few;
    static_cast<Common&>(few) = l;
    for (int i = 0; i < l.count; ++i) few.t[i] = l.t[i];
    launch_size<PT, GT, MASTER>(eight, tiles, few, s);
  } else {
    launch_size<PT, GT, MASTER>(eight, tiles, l, s);
  }
}

template <typename PT>
void launch_typed(const ftmoe_adamw_tensor& like, uint32_t tiles, const Launch<kMaxTensors>& l, cudaStream_t s) {
  const bool eight = like.state_bits == 8, wide = like.g_dtype == FTMOE_FP32, master = like.master != nullptr;
  if constexpr (std::is_same<PT, float>::value) {
    launch_kind<float, float, false>(eight, tiles, l, s);
  } else if (master) {
    if (wide) launch_kind<PT, float, true>(eight, tiles, l, s);
    else launch_kind<PT, PT, true>(eight, tiles, l, s);
  } else {
    if (wide) launch_kind<PT, float, false>(eight, tiles, l, s);
    else launch_kind<PT, PT, false>(eight, tiles, l, s);
  }
}

// Tensors of one kind share a launch.
inline int kind_of(const ftmoe_adamw_tensor& t) {
  return t.p_dtype | t.g_dtype << 2 | (t.master ? 16 : 0) | (t.state_bits == 8 ? 32 : 0);
}

inline uint32_t aligned(const ftmoe_adamw_tensor& t) {
  return (((uintptr_t)t.p | (uintptr_t)t.g | (uintptr_t)t.master) & 15) == 0 &&
         (((uintptr_t)t.m | (uintptr_t)t.v) & 7) == 0;
}

}  // namespace

cudaError_t launch_adamw(const TrainDevice& d, const ftmoe_adamw_tensor* list, int n, const ftmoe_adamw_params& hp,
                         cudaStream_t s) {
  Launch<kMaxTensors> l;
  l.b1 = (float)hp.beta1;
  l.ob1 = (float)(1.0 - hp.beta1);
  l.b2 = (float)hp.beta2;
  l.ob2 = (float)(1.0 - hp.beta2);
  l.root_scale = (float)(1.0 / std::sqrt(1.0 - std::pow(hp.beta2, (double)hp.step)));
  l.eps = (float)hp.eps;
  l.lr = (float)(hp.lr / (1.0 - std::pow(hp.beta1, (double)hp.step)));
  l.grad_scale = hp.grad_scale;
  uint64_t kinds = 0;
  for (int i = 0; i < n; ++i) kinds |= list[i].n ? 1ull << kind_of(list[i]) : 0;
  for (int kind = 0; kind < 64; ++kind) {
    if (!(kinds >> kind & 1)) continue;
    l.count = 0;
    // short tiles until there are enough of them to fill the SMs four times
    int64_t blocks = 0;
    for (int i = 0; i < n; ++i)
      if (list[i].n && kind_of(list[i]) == kind) blocks += (list[i].n + 255) / 256;
    l.tile_blocks = (int)std::clamp<int64_t>(blocks / ((int64_t)d.num_sms * 32 * 4), 1, kMaxTileBlocks);
    uint32_t tiles = 0;
    const ftmoe_adamw_tensor* like = nullptr;
    auto flush = [&]() {
      if (l.count) with_dtype(like->p_dtype, [&](auto type) {
        launch_typed<decltype(type)>(*like, tiles, l, s);
        return cudaSuccess;
      });
      l.count = 0;
      tiles = 0;
      return cudaGetLastError();
    };
    for (int i = 0; i < n; ++i) {
      const ftmoe_adamw_tensor& t = list[i];
      if (t.n == 0 || kind_of(t) != kind) continue;
      const int64_t tile = t.state_bits == 8 ? l.tile_blocks * 256 : kTile, need = (t.n + tile - 1) / tile;
      if (l.count == kMaxTensors || tiles + need > INT32_MAX) {
        const cudaError_t e = flush();
        if (e != cudaSuccess) return e;
      }
      like = &t;
      l.t[l.count++] = {t.p, t.g, t.master, t.m, t.v, t.m_scale, t.v_scale, t.n, tiles,
                        (float)(1.0 - hp.lr * t.weight_decay), aligned(t)};
      tiles += (uint32_t)need;
    }
    const cudaError_t e = flush();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ftmoe
