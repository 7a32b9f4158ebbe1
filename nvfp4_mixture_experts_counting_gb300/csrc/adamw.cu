// One AdamW step over many tensors, with states in 32 bits or in 8.
//
// With g' = grad_scale * g and t the step's number from 1:
//   m <- b1 m + (1 - b1) g',  v <- b2 v + (1 - b2) g'^2
//   p <- p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32, each operation rounded on its own (no contraction), so that the
// 8-bit codes below are those of the formula, bit for bit.
//
// 8 bits: m and the root u = sqrt(v) are E4M3 codes with one fp32 scale for
// each 256 values of the tensor, scale = amax * fl(1/448), code = E4M3(x *
// (448 * fl(1/amax))).  The root and not v is held: its codes then span 2^17
// in u, 2^34 in v, and the update divides by u.  A root that is not zero never rounds to zero, which would make the next
// step's divisor eps alone.
#include <cmath>

#include "train_common.cuh"

namespace ftmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                  // values a thread updates
constexpr int kTile = kThreads * kPer;   // a warp's 256 values are one 8-bit block
// Tensors of one launch: the descriptors travel as kernel parameters, and
// 29 KB of them cost some 3 us of the launch, so short lists have a kernel of their own.
constexpr int kFewTensors = 24, kMaxTensors = 400;
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
};

struct Common {
  float b1, ob1, b2, ob2, root_scale, eps, lr;
  const float* grad_scale;
  int count;
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

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t i, int64_t n, float scale, float (&f)[kPer]) {
  uint32_t w[2] = {0, 0};
  if (i + kPer <= n && ((uintptr_t)(p + i) & 7) == 0) {
    const uint2 r = *reinterpret_cast<const uint2*>(p + i);
    w[0] = r.x;
    w[1] = r.y;
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (i + c < n) w[c / 4] |= (uint32_t)p[i + c] << (c % 4 * 8);
  }
#pragma unroll
  for (int c = 0; c < kPer; c += 2) {
    uint32_t h;
    const uint16_t in = (uint16_t)(w[c / 4] >> (c % 4 * 8));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
    const float2 d = __half22float2(*reinterpret_cast<__half2*>(&h));
    f[c] = __fmul_rn(d.x, scale);
    f[c + 1] = __fmul_rn(d.y, scale);
  }
}

// Codes of a warp's block; returns its scale.  FLOOR: values above zero keep the smallest code.
template <bool FLOOR>
__device__ __forceinline__ float store_codes(uint8_t* p, int64_t i, int64_t n, const float (&f)[kPer]) {
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < kPer; ++c) top = fmaxf(top, fabsf(f[c]));
  top = warp_max_f32(top);
  const bool flat = top < kTiny;
  const float r = flat ? 0.f : __fmul_rn(__frcp_rn(top), 448.f);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < kPer; c += 2) {
    uint32_t q = e4m3x2(__fmul_rn(f[c], r), __fmul_rn(f[c + 1], r));
    if (FLOOR && !flat) {
      if ((q & 0xff) == 0 && f[c] > 0.f) q |= 1;
      if ((q & 0xff00) == 0 && f[c + 1] > 0.f) q |= 0x100;
    }
    w[c / 4] |= q << (c % 4 * 8);
  }
  if (i + kPer <= n && ((uintptr_t)(p + i) & 7) == 0) {
    *reinterpret_cast<uint2*>(p + i) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (i + c < n) p[i + c] = (uint8_t)(w[c / 4] >> (c % 4 * 8));
  }
  return flat ? 0.f : __fmul_rn(top, 1.f / 448.f);
}

template <typename PT, typename GT, bool MASTER, bool EIGHT, int CAP>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ Launch<CAP> a) {
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  if (!isfinite(gs)) return;  // an overflowed step is skipped
  int lo = 0, hi = a.count - 1;  // the last tensor that starts at or before this tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].tile0 <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const Tensor& t = a.t[lo];
  const int64_t i = (int64_t)(blockIdx.x - t.tile0) * kTile + threadIdx.x * kPer, n = t.n;
  const int64_t block = i / 256;
  if (block * 256 >= n) return;  // a whole warp's block lies past the tensor
  float p[kPer], g[kPer], m[kPer], v[kPer], u[kPer];
  load8(static_cast<const GT*>(t.g), i, n, g);
  if (MASTER) load8(static_cast<const float*>(t.master), i, n, p);
  else load8(static_cast<const PT*>(t.p), i, n, p);
  if (EIGHT) {
    load_codes(static_cast<const uint8_t*>(t.m), i, n, t.m_scale[block], m);
    load_codes(static_cast<const uint8_t*>(t.v), i, n, t.v_scale[block], v);
#pragma unroll
    for (int c = 0; c < kPer; ++c) v[c] = __fmul_rn(v[c], v[c]);
  } else {
    load8(static_cast<const float*>(t.m), i, n, m);
    load8(static_cast<const float*>(t.v), i, n, v);
  }
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const float gc = __fmul_rn(g[c], gs);
    m[c] = __fadd_rn(__fmul_rn(m[c], a.b1), __fmul_rn(gc, a.ob1));
    v[c] = __fadd_rn(__fmul_rn(v[c], a.b2), __fmul_rn(__fmul_rn(gc, gc), a.ob2));
    u[c] = __fsqrt_rn(v[c]);
    const float update = __fdiv_rn(m[c], __fadd_rn(__fmul_rn(u[c], a.root_scale), a.eps));
    p[c] = __fsub_rn(__fmul_rn(p[c], t.decay), __fmul_rn(update, a.lr));
  }
  store8(static_cast<PT*>(t.p), i, n, p);
  if (MASTER) store8(t.master, i, n, p);
  if (EIGHT) {
    const float ms = store_codes<false>(static_cast<uint8_t*>(t.m), i, n, m);
    const float us = store_codes<true>(static_cast<uint8_t*>(t.v), i, n, u);
    if ((threadIdx.x & 31) == 0) {
      t.m_scale[block] = ms;
      t.v_scale[block] = us;
    }
  } else {
    store8(static_cast<float*>(t.m), i, n, m);
    store8(static_cast<float*>(t.v), i, n, v);
  }
}

template <typename PT, typename GT, bool MASTER>
void launch_kind(bool eight, uint32_t tiles, const Launch<kMaxTensors>& l, cudaStream_t s) {
  if (l.count <= kFewTensors) {
    Launch<kFewTensors> few;
    static_cast<Common&>(few) = l;
    for (int i = 0; i < l.count; ++i) few.t[i] = l.t[i];
    if (eight) k_adamw<PT, GT, MASTER, true, kFewTensors><<<tiles, kThreads, 0, s>>>(few);
    else k_adamw<PT, GT, MASTER, false, kFewTensors><<<tiles, kThreads, 0, s>>>(few);
  } else {
    if (eight) k_adamw<PT, GT, MASTER, true, kMaxTensors><<<tiles, kThreads, 0, s>>>(l);
    else k_adamw<PT, GT, MASTER, false, kMaxTensors><<<tiles, kThreads, 0, s>>>(l);
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

}  // namespace

cudaError_t launch_adamw(const ftmoe_adamw_tensor* list, int n, const ftmoe_adamw_params& hp, cudaStream_t s) {
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
      const int64_t need = (t.n + kTile - 1) / kTile;
      if (l.count == kMaxTensors || tiles + need > INT32_MAX) {
        const cudaError_t e = flush();
        if (e != cudaSuccess) return e;
      }
      like = &t;
      l.t[l.count++] = {t.p, t.g, t.master, t.m, t.v, t.m_scale, t.v_scale, t.n, tiles,
                        (float)(1.0 - hp.lr * t.weight_decay)};
      tiles += (uint32_t)need;
    }
    const cudaError_t e = flush();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ftmoe
