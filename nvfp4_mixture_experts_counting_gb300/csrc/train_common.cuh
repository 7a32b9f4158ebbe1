// Device helpers of the training operators: rows of bf16, fp16 or fp32 values
// read and written 16 bytes (or one value) at a time, with the arithmetic in fp32.
#pragma once

#include "common.cuh"
#include "tma.cuh"
#include "train.h"

namespace ftmoe {

inline int dtype_bytes(int dtype) { return dtype == FTMOE_FP32 ? 4 : 2; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// The unsigned type of an access of B bytes.
template <int B> struct Raw;
template <> struct Raw<2> { using type = uint16_t; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };

// N values of T moved in one access.
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
  T v[N];
  __device__ __forceinline__ float get(int i) const { return to_f32(v[i]); }
  __device__ __forceinline__ void set(int i, float f) { v[i] = from_f32<T>(f); }
};

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* p) {
  constexpr int B = sizeof(T) * N < 16 ? sizeof(T) * N : 16;  // of one access; 32 bytes take two
  using R = typename Raw<B>::type;
  Pack<T, N> v;
#pragma unroll
  for (int i = 0; i < (int)sizeof(v) / B; ++i) reinterpret_cast<R*>(&v)[i] = reinterpret_cast<const R*>(p)[i];
  return v;
}
template <typename T, int N>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, N>& v) {
  constexpr int B = sizeof(T) * N < 16 ? sizeof(T) * N : 16;
  using R = typename Raw<B>::type;
#pragma unroll
  for (int i = 0; i < (int)sizeof(v) / B; ++i) reinterpret_cast<R*>(p)[i] = reinterpret_cast<const R*>(&v)[i];
}

// i / n, in 32 bits where that holds it.
__device__ __forceinline__ int64_t quotient(int64_t i, int n) {
  return i >> 32 ? i / n : (int64_t)((uint32_t)i / (uint32_t)n);
}

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max_f32(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Two fp32 values in one 64-bit register, and the packed arithmetic on them.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Values 2e and 2e + 1 of a piece as fp32, and back.
template <int N>
__device__ __forceinline__ uint64_t pair_of(const Pack<float, N>& x, int e) {
  return pack2(x.v[2 * e], x.v[2 * e + 1]);
}
template <int N>
__device__ __forceinline__ uint64_t pair_of(const Pack<__nv_bfloat16, N>& x, int e) {
  const uint32_t b = reinterpret_cast<const uint32_t*>(&x)[e];
  return pack2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
}
template <int N>
__device__ __forceinline__ uint64_t pair_of(const Pack<__half, N>& x, int e) {
  const float2 f = __half22float2(reinterpret_cast<const __half2*>(&x)[e]);
  return pack2(f.x, f.y);
}
template <int N>
__device__ __forceinline__ void set_pair(Pack<float, N>& o, int e, uint64_t v) {
  unpack2(v, o.v[2 * e], o.v[2 * e + 1]);
}
template <int N>
__device__ __forceinline__ void set_pair(Pack<__nv_bfloat16, N>& o, int e, uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  reinterpret_cast<__nv_bfloat162*>(&o)[e] = __floats2bfloat162_rn(lo, hi);
}
template <int N>
__device__ __forceinline__ void set_pair(Pack<__half, N>& o, int e, uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  reinterpret_cast<__half2*>(&o)[e] = __floats2half2_rn(lo, hi);
}

// Shared -> global bulk copy (16-byte aligned, a multiple of 16 bytes), and the
// wait until the sources of all but the last PENDING groups may be overwritten.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(PENDING) : "memory");
}

// This thread's accesses to shared memory before, asynchronous copies' after.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Launches a kernel that calls pdl_wait before it uses what the stream's
// previous kernel writes: it may start while that one ends.
template <typename... A, typename... B>
cudaError_t launch_after_smem(void (*k)(A...), unsigned grid, int threads, size_t smem, cudaStream_t s, B... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, static_cast<A>(args)...);
}
template <typename... A, typename... B>
cudaError_t launch_after(void (*k)(A...), unsigned grid, int threads, cudaStream_t s, B... args) {
  return launch_after_smem(k, grid, threads, 0, s, args...);
}

// Calls f with a value of the type that a dtype code names.
template <typename F>
cudaError_t with_dtype(int dtype, F f) {
  if (dtype == FTMOE_FP32) return f(float());
  if (dtype == FTMOE_FP16) return f(__half());
  return f(__nv_bfloat16());
}

}  // namespace ftmoe
