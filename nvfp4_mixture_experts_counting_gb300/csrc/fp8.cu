// E4M3 quantisers of activations (a scale for 128 values) and weights (for 128
// x 128), and SwiGLU between two products with its gradient.
//
// All are one pass over their data, bound by DRAM: eight lanes hold a block of
// 128 values, 16 each, so that a lane reads 32 bytes (64 of fp32) and writes
// its 16 codes in one store, and a block's largest magnitude takes three
// shuffles.
#include "fp8_common.cuh"

namespace ftmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;  // of a block
constexpr int kPer = kFp8Block / kLanes;

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[kPer]) {
  constexpr int N = 16 / sizeof(T);
  Pack<T, N> x[kPer / N];
#pragma unroll
  for (int i = 0; i < kPer / N; ++i) x[i] = load_pack<T, N>(p + i * N);
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = x[i / N].get(i % N);
}

// The scale of the block that this lane's group of eight holds, and this lane's codes.
__device__ __forceinline__ uint4 quantize16(const float (&v)[kPer], float& scale) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) most = max_magnitude(most, v[i]);
  uint32_t top = magnitude(most);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const BlockScale b = block_scale(top);
  scale = b.scale;
  if (b.mul == 0.f && b.scale == 0.f) return make_uint4(0, 0, 0, 0);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3x4(v[4 * i] * b.mul, v[4 * i + 1] * b.mul, v[4 * i + 2] * b.mul, v[4 * i + 3] * b.mul);
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// A warp takes eight neighbouring blocks of a row, two at each lane's place
// whose loads go out together.  With `inv`, token t's codes go to the rows
// inv[t * top_k + j].
//
// 16384 tokens of 2560 bf16 values to eight rows each: 76 us, 5.7 TB/s of a
// copy's 6.8.  Most of the rest is the scales: 4 bytes to a line of its own for
// each block and row, which every lane writes (by one lane in eight 79 us; not
// at all some 66).  Grids of up to 64 CTAs an SM, so that few warps come round
// the loop.
constexpr int kTwice = 2;
template <typename T>
__global__ void __launch_bounds__(kThreads) k_fp8_quantize(const T* x, int T_, int K, const int32_t* inv, int top_k,
                                                           const int32_t* used, uint8_t* codes, float* scales,
                                                           uint32_t* status) {
  pdl_wait();
  const int rows = used_rows(used, T_, status);
  const int64_t places = inv ? (int64_t)T_ * top_k : T_;
  const int blocks = (K + kFp8Block - 1) / kFp8Block, parts = (blocks + 4 * kTwice - 1) / (4 * kTwice);
  const int lane = threadIdx.x & 31, sub = lane & (kLanes - 1);
  const int64_t units = (int64_t)rows * parts, step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; u < units; u += step) {
    const int64_t t = quotient(u, parts);
    const int b0 = (int)(u - t * parts) * (4 * kTwice) + lane / kLanes;
    int mine = -1;
    if (inv && lane < top_k) {
      mine = inv[t * top_k + lane];
      if (mine < -1 || mine >= places) {
        set_status(status, kStatusRange);
        mine = -1;
      }
    }
    float v[kTwice][kPer];
#pragma unroll
    for (int h = 0; h < kTwice; ++h) {
      const int k0 = (b0 + 4 * h) * kFp8Block + sub * kPer;
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[h][i] = 0.f;
      if (k0 < K) load16(x + t * K + k0, v[h]);  // K is a multiple of 16: a lane's values are all there or none is
    }
    uint4 c[kTwice];
    float scale[kTwice];
#pragma unroll
    for (int h = 0; h < kTwice; ++h) c[h] = quantize16(v[h], scale[h]);
    for (int j = 0; j < top_k; ++j) {
      const int64_t at = inv ? __shfl_sync(0xffffffffu, mine, j) : t;
      if (at < 0) continue;
#pragma unroll
      for (int h = 0; h < kTwice; ++h) {
        const int k0 = (b0 + 4 * h) * kFp8Block + sub * kPer;
        if (k0 < K) *reinterpret_cast<uint4*>(codes + at * K + k0) = c[h];
      }
    }
    // The scales, each to a line of its own: lane l those of block l % 8, of every fourth place.
    static_assert(kTwice == 2 && kLanes == 8, "eight blocks a warp");
    const float s0 = __shfl_sync(0xffffffffu, scale[0], (lane & 3) * kLanes);
    const float s1 = __shfl_sync(0xffffffffu, scale[1], (lane & 3) * kLanes);
    const int b = (int)(u - t * parts) * 8 + (lane & 7);
    for (int j = lane >> 3; j < (top_k + 3 & ~3); j += 4) {
      const int to = __shfl_sync(0xffffffffu, mine, j & 31);
      const int64_t at = inv ? (int64_t)to : t;
      if (j < top_k && at >= 0 && b < blocks) scales[(int64_t)b * places + at] = lane & 4 ? s1 : s0;
    }
  }
}

// A CTA takes a block of 128 x 128, a row of it per 8 lanes, and reads it again
// (from L1 or L2) once its scale is known.  A load-time tool, bound by DRAM: 64
// matrices of 1280 x 2560 from bf16 103 us, 6.1 TB/s; from fp32 200 us, 5.2 TB/s.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_fp8_quantize_weights(const T* w, int N, int K, uint8_t* codes,
                                                                   float* scales) {
  __shared__ uint32_t part[kThreads / 32];
  const int blocks = (K + kFp8Block - 1) / kFp8Block, kb = blockIdx.x % blocks, nb = blockIdx.x / blocks;
  const int64_t e = blockIdx.y;
  const int sub = threadIdx.x % kLanes, k0 = kb * kFp8Block + sub * kPer;
  constexpr int kRows = kThreads / kLanes;
  uint32_t top = 0;
  for (int r = threadIdx.x / kLanes; r < kFp8Block; r += kRows) {
    const int n = nb * kFp8Block + r;
    if (n >= N || k0 >= K) continue;
    float v[kPer];
    load16(w + (e * N + n) * K + k0, v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) top = max(top, magnitude(v[i]));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) top = max(top, part[i]);
  const BlockScale b = block_scale(top);
  if (threadIdx.x == 0) scales[e * gridDim.x + blockIdx.x] = b.scale;
  for (int r = threadIdx.x / kLanes; r < kFp8Block; r += kRows) {
    const int n = nb * kFp8Block + r;
    if (n >= N || k0 >= K) continue;
    float v[kPer];
    load16(w + (e * N + n) * K + k0, v);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = b.scale == 0.f ? 0u : e4m3x4(v[4 * i] * b.mul, v[4 * i + 1] * b.mul, v[4 * i + 2] * b.mul, v[4 * i + 3] * b.mul);
    *reinterpret_cast<uint4*>(codes + (e * N + n) * K + k0) = make_uint4(c[0], c[1], c[2], c[3]);
  }
}

// ---------------------------------------------------------------- SwiGLU

// h = g s(g) u, and its gradient from dh: dg = dh u s (1 + g (1 - s)), du = dh g s.
__device__ __forceinline__ float swiglu(float g, float u) { return g * sigmoid_rcp(g) * u; }
__device__ __forceinline__ void swiglu_grad(float dh, float g, float u, float& dg, float& du) {
  const float s = sigmoid_rcp(g);
  dg = dh * u * s * (1.f + g * (1.f - s));
  du = dh * g * s;
}

// Quantised output: eight lanes take 128 columns of a row.  GRAD writes a row
// of 2 I codes, gate's first.  131072 x 640 from bf16: 79 us, 5.3 TB/s, the issue
// slots busiest with the exponentials' instructions (104 us with a division in
// the sigmoid instead of the approximate reciprocal; its gradient to codes 151
// instead of 116 us, 5.8 TB/s).
template <typename T, bool GRAD>
__global__ void __launch_bounds__(kThreads) k_swiglu_fp8(const T* gu, const T* dh, int rows_, int I,
                                                         const int32_t* used, uint8_t* codes, float* scales,
                                                         uint32_t* status) {
  pdl_wait();
  const int rows = used_rows(used, rows_, status), blocks = I / kFp8Block;
  const int sub = threadIdx.x % kLanes;
  const int64_t units = (int64_t)rows * blocks, step = (int64_t)gridDim.x * (kThreads / kLanes);
  // whole warps leave the loop together: the shuffles need all lanes
  for (int64_t u0 = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / 32 * 4; u0 < units; u0 += step) {
    const int64_t u = u0 + (threadIdx.x & 31) / kLanes;
    const bool on = u < units;
    const int64_t r = on ? quotient(u, blocks) : 0;
    const int b = on ? (int)(u - r * blocks) : 0, k0 = b * kFp8Block + sub * kPer;
    float g[kPer], v[kPer];
    load16(gu + r * 2 * I + k0, g);
    load16(gu + r * 2 * I + I + k0, v);
    float scale;
    if constexpr (GRAD) {
      float d[kPer];
      load16(dh + r * I + k0, d);
#pragma unroll
      for (int i = 0; i < kPer; ++i) swiglu_grad(d[i], g[i], v[i], g[i], v[i]);
      const uint4 cg = quantize16(g, scale);
      if (on) {
        *reinterpret_cast<uint4*>(codes + r * 2 * I + k0) = cg;
        if (sub == 0) scales[(int64_t)b * rows_ + r] = scale;
      }
      const uint4 cu = quantize16(v, scale);
      if (on) {
        *reinterpret_cast<uint4*>(codes + r * 2 * I + I + k0) = cu;
        if (sub == 0) scales[(int64_t)(blocks + b) * rows_ + r] = scale;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = swiglu(g[i], v[i]);
      const uint4 c = quantize16(v, scale);
      if (on) {
        *reinterpret_cast<uint4*>(codes + r * I + k0) = c;
        if (sub == 0) scales[(int64_t)b * rows_ + r] = scale;
      }
    }
  }
}

// Output in the input's type.  A warp takes neighbouring pieces of a row, a
// lane one (or four, 32 pieces apart) of V = 16 bytes' values, or of one value
// where rows are not a multiple of 16 bytes.  Four where a lane has little on
// its way otherwise (the gradient of 8191 x 1001 fp16 values 19 us, 28 with
// one); with two 16-byte loads a lane more warps at a time are better (131072 x
// 640 bf16 values 84 us, 96 with four).  The gradient of whole 16 bytes has four:
// of 65536 x 1024 bf16 values 98 us (one: 108), 131072 x 2048 388 (424), 131072 x
// 640 fp16 125 (139), bf16 141 (138); it loses where rows are shorter than the
// four pieces' 1024 values (262144 x 256 bf16 155 us, one 108).  Two lie between.
template <int V, bool GRAD>
constexpr int kPieces = V > 1 && !GRAD ? 1 : 4;
template <typename T, int V, bool GRAD>
__global__ void __launch_bounds__(kThreads) k_swiglu(const T* gu, const T* dh, int rows_, int I, const int32_t* used,
                                                     T* out, uint32_t* status) {
  pdl_wait();
  constexpr int kN = kPieces<V, GRAD>, kWide = 32 * V * kN;
  const int rows = used_rows(used, rows_, status), chunks = (I + kWide - 1) / kWide;
  const int64_t units = (int64_t)rows * chunks, step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; i < units; i += step) {
    const int64_t r = quotient(i, chunks);
    const int k0 = (int)(i - r * chunks) * kWide + (threadIdx.x & 31) * V;
    const T *g = gu + r * 2 * I, *u = g + I, *d = GRAD ? dh + r * I : nullptr;
    T* o = out + r * (GRAD ? 2 : 1) * I;
    Pack<T, V> pg[kN], pu[kN], pd[kN];
#pragma unroll
    for (int p = 0; p < kN; ++p) {
      const int k = k0 + 32 * V * p;
      if (k >= I) continue;
      pg[p] = load_pack<T, V>(g + k);
      pu[p] = load_pack<T, V>(u + k);
      if (GRAD) pd[p] = load_pack<T, V>(d + k);
    }
#pragma unroll
    for (int p = 0; p < kN; ++p) {
      const int k = k0 + 32 * V * p;
      if (k >= I) continue;
      Pack<T, V> a, b;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (GRAD) {
          float dg, du;
          swiglu_grad(pd[p].get(j), pg[p].get(j), pu[p].get(j), dg, du);
          a.set(j, dg);
          b.set(j, du);
        } else {
          a.set(j, swiglu(pg[p].get(j), pu[p].get(j)));
        }
      }
      store_pack<T, V>(o + k, a);
      if (GRAD) store_pack<T, V>(o + I + k, b);
    }
  }
}

unsigned grid_of(const TrainDevice& d, int64_t work, int per_cta, int ctas_per_sm) {
  const int64_t need = (work + per_cta - 1) / per_cta, most = (int64_t)d.num_sms * ctas_per_sm;
  return (unsigned)(need < 1 ? 1 : need < most ? need : most);
}

}  // namespace

cudaError_t launch_fp8_quantize(const TrainDevice& d, const void* x, int dtype, int T, int K, const int32_t* inv,
                                int top_k, const int32_t* used, uint8_t* codes, float* scales, cudaStream_t s) {
  return with_dtype(dtype, [&](auto zero) {
    using V = decltype(zero);
    const int64_t units = (int64_t)T * ((fp8_blocks(K) + 4 * kTwice - 1) / (4 * kTwice));
    return launch_after(k_fp8_quantize<V>, grid_of(d, units, kThreads / 32, 64), kThreads, s,
                        static_cast<const V*>(x), T, K, inv, top_k, used, codes, scales, d.status);
  });
}

cudaError_t launch_fp8_quantize_weights(const TrainDevice& d, const void* w, int dtype, int E, int N, int K,
                                        uint8_t* codes, float* scales, cudaStream_t s) {
  return with_dtype(dtype, [&](auto zero) {
    using V = decltype(zero);
    const dim3 grid((unsigned)fp8_blocks(K) * fp8_blocks(N), E);
    k_fp8_quantize_weights<V><<<grid, kThreads, 0, s>>>(static_cast<const V*>(w), N, K, codes, scales);
    return cudaGetLastError();
  });
}

cudaError_t launch_swiglu(const TrainDevice& d, const void* gu, const void* dh, int dtype, int rows, int I,
                          const int32_t* used, void* out, float* scales, cudaStream_t s) {
  return with_dtype(dtype, [&](auto zero) {
    using V = decltype(zero);
    const V *g = static_cast<const V*>(gu), *dv = static_cast<const V*>(dh);
    if (scales) {
      const unsigned grid = grid_of(d, (int64_t)rows * (I / kFp8Block), kThreads / kLanes, 16);
      return launch_after(dh ? k_swiglu_fp8<V, true> : k_swiglu_fp8<V, false>, grid, kThreads, s, g, dv, rows, I, used,
                          static_cast<uint8_t*>(out), scales, d.status);
    }
    constexpr int W = 16 / sizeof(V);
    const bool wide = I % W == 0;
    const int per_warp = 32 * (wide ? W * (dh ? kPieces<W, true> : kPieces<W, false>) : kPieces<1, true>);
    const unsigned grid = grid_of(d, (int64_t)rows * ((I + per_warp - 1) / per_warp), kThreads / 32, 16);
    auto* k = wide ? (dh ? k_swiglu<V, W, true> : k_swiglu<V, W, false>)
                   : (dh ? k_swiglu<V, 1, true> : k_swiglu<V, 1, false>);
    return launch_after(k, grid, kThreads, s, g, dv, rows, I, used, static_cast<V*>(out), d.status);
  });
}

}  // namespace ftmoe
