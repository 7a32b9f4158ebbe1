// Product of E4M3 codes with a scale for each block of 128, grouped by expert:
//   y[r, n] = sum_b sx[b, r] sw[n / 128, b] sum_{k in block b} qx[r, k] qw[n, k]
// and with `transpose` the product with the weights' columns (the gradient of
// the input), or with `swiglu` h = SwiGLU of y's halves as codes and scales.
#include "fp8_common.cuh"

namespace ftmoe {

namespace {

// The rows of expert e, none where they begin before an earlier expert's end
// (`floor`, kept along), fall or leave [0, M]; that marks the status word.
__device__ __forceinline__ int2 expert_rows(const int32_t* offsets, int e, int M, int& floor, uint32_t* status) {
  if (!offsets) return make_int2(0, M);
  const int lo = offsets[e], hi = offsets[e + 1];
  const bool good = lo >= floor && hi >= lo && hi <= M;
  floor = max(floor, lo);
  if (good) return make_int2(lo, hi);
  set_status(status, kStatusRange);
  return make_int2(0, 0);
}

constexpr int kRows = 8;  // of a tile

struct MatmulArgs {
  const uint8_t *a, *w;
  const float *a_scale, *w_scale;
  const int32_t* offsets;
  int M, E, N, K, transpose, swiglu, dtype;
  void* out;
  float* out_scale;
  uint32_t* status;
};

__device__ __forceinline__ void store_out(void* out, int dtype, int64_t i, float v) {
  if (dtype == FTMOE_FP32) static_cast<float*>(out)[i] = v;
  else if (dtype == FTMOE_FP16) static_cast<__half*>(out)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

// A thread computes kRows tokens of one output column (with SwiGLU of a gate
// and an up column).
__global__ void __launch_bounds__(128) k_fp8_matmul_plain(const __grid_constant__ MatmulArgs a) {
  __shared__ float xs[kRows][kFp8Block];
  __shared__ uint32_t tops[kRows][4];
  const int C = a.transpose ? a.N : a.K, O = a.transpose ? a.K : a.swiglu ? a.N / 2 : a.N;
  const int CB = (C + 127) / 128, KB = (a.K + 127) / 128, NB = (a.N + 127) / 128;
  const int o = blockIdx.y * 128 + threadIdx.x;
  int tile = blockIdx.x, e = 0, floor = 0;
  uint32_t* status = threadIdx.x == 0 ? a.status : nullptr;
  int2 r = make_int2(0, 0);
  for (; e < a.E; ++e) {
    r = expert_rows(a.offsets, e, a.M, floor, status);
    const int n = (r.y - r.x + kRows - 1) / kRows;
    if (tile < n) break;
    tile -= n;
  }
  if (e == a.E) return;
  const int row0 = r.x + tile * kRows, rows = min(kRows, r.y - row0);
  const int64_t bank = (int64_t)e * a.N * a.K;
  float acc[2][kRows] = {};
  for (int b = 0; b < CB; ++b) {
    const int c0 = b * 128, len = min(128, C - c0);
    __syncthreads();
    for (int i = 0; i < rows; ++i)
      xs[i][threadIdx.x] =
          threadIdx.x < len ? e4m3_decode(a.a[(int64_t)(row0 + i) * C + c0 + threadIdx.x]) : 0.f;
    __syncthreads();
    if (o >= O) continue;
    for (int half = 0; half < (a.swiglu ? 2 : 1); ++half) {
      const int n = o + half * O;
      float d[kRows] = {};
      for (int k = 0; k < len; ++k) {
        const int64_t at = a.transpose ? (int64_t)(c0 + k) * a.K + n : (int64_t)n * a.K + c0 + k;
        const float w = e4m3_decode(a.w[bank + at]);
        for (int i = 0; i < kRows; ++i) d[i] += w * xs[i][k];
      }
      const float sw = a.w_scale[((int64_t)e * NB + (a.transpose ? b : n / 128)) * KB + (a.transpose ? n / 128 : b)];
      for (int i = 0; i < rows; ++i) acc[half][i] += d[i] * (a.a_scale[(int64_t)b * a.M + row0 + i] * sw);
    }
  }
  if (!a.swiglu) {
    if (o < O)
      for (int i = 0; i < rows; ++i) store_out(a.out, a.dtype, (int64_t)(row0 + i) * O + o, acc[0][i]);
    return;
  }
  for (int i = 0; i < rows; ++i) {
    acc[0][i] = acc[0][i] * sigmoid(acc[0][i]) * acc[1][i];
    const uint32_t top = __reduce_max_sync(0xffffffffu, magnitude(acc[0][i]));
    if (threadIdx.x % 32 == 0) tops[i][threadIdx.x / 32] = top;
  }
  __syncthreads();
  for (int i = 0; i < rows; ++i) {
    const BlockScale s = block_scale(max(max(tops[i][0], tops[i][1]), max(tops[i][2], tops[i][3])));
    const float v = s.scale == 0.f ? 0.f : acc[0][i] * s.mul;
    static_cast<uint8_t*>(a.out)[(int64_t)(row0 + i) * O + o] = (uint8_t)e4m3x4(v, 0.f, 0.f, 0.f);
    if (threadIdx.x == 0) a.out_scale[(int64_t)blockIdx.y * a.M + row0 + i] = s.scale;
  }
}

}  // namespace

cudaError_t launch_fp8_matmul(const TrainDevice& d, const ftmoe_fp8_matmul_args& m, cudaStream_t s) {
  const MatmulArgs a{m.a, m.w, m.a_scale, m.w_scale, m.offsets, (int)m.M, m.E, m.N, m.K, m.transpose, m.swiglu,
                     m.out_dtype, m.out, m.out_scale, d.status};
  const int O = m.transpose ? m.K : m.swiglu ? m.N / 2 : m.N;
  const dim3 grid((unsigned)(m.M / kRows + m.E), (unsigned)fp8_blocks(O));
  k_fp8_matmul_plain<<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ftmoe
