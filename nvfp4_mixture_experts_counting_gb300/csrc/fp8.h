// Host-side declarations of the 8-bit layer's kernel launchers (internal):
// routing from logits, quantisers, the grouped product and SwiGLU.
#pragma once

#include "train.h"

namespace ftmoe {

constexpr int kFp8Block = 128;      // values that share one scale; of weights 128 x 128 do
constexpr float kFp8Max = 448.f;    // the largest E4M3 value
constexpr float kFp8Tiny = 1e-30f;  // a block whose largest magnitude is below this is held as zeros
constexpr int kMaxGroups = 32;      // of experts, in routing

inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

// The current device, set up once (train.cu).
int train_device(TrainDevice* out);

// Routing (route_topk.cu).
cudaError_t launch_route_topk(const TrainDevice& d, const ftmoe_route_args& a, cudaStream_t s);
cudaError_t launch_route_topk_backward(const TrainDevice& d, const ftmoe_route_args& a, const float* dw, void* dlogits,
                                       int64_t ld_d, cudaStream_t s);

// Quantisers and SwiGLU (fp8.cu).
cudaError_t launch_fp8_quantize(const TrainDevice& d, const void* x, int dtype, int T, int K, const int32_t* inv,
                                int top_k, const int32_t* used, uint8_t* codes, float* scales, cudaStream_t s);
cudaError_t launch_fp8_quantize_weights(const TrainDevice& d, const void* w, int dtype, int E, int N, int K,
                                        uint8_t* codes, float* scales, cudaStream_t s);
cudaError_t launch_swiglu(const TrainDevice& d, const void* gu, const void* dh, int dtype, int rows, int I,
                          const int32_t* used, void* out, float* scales, cudaStream_t s);

// Grouped product (fp8_matmul.cu).
cudaError_t fp8_matmul_set_limits();
cudaError_t launch_fp8_matmul(const TrainDevice& d, const ftmoe_fp8_matmul_args& a, cudaStream_t s);

}  // namespace ftmoe
