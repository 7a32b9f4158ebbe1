// Host-side declarations of the training operators' kernel launchers
// (internal): tokens sorted by expert and back, embedding, policy loss, AdamW.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ftmoe.h"

namespace ftmoe {

// What a launcher needs to know of the current device.
struct TrainDevice {
  uint32_t* status;  // device word that the operators' range checks mark
  int num_sms;
  int sort_ctas;  // CTAs of the cluster that sorts
  uint32_t test_wait_ns;    // ftmoe_test_withhold_policy's limit, or 0
  uint32_t test_matmul_ns;  // ftmoe_test_withhold_matmul's
};

constexpr int kMaxBins = 1024;  // experts, or values of one radix digit
constexpr int kSortCtas = 16;   // CTAs of the cluster that sorts, at most (8 is the portable limit)

// Tokens sorted by expert and back (dispatch.cu).
cudaError_t dispatch_set_limits(int* sort_ctas);
cudaError_t launch_dispatch(const TrainDevice& d, const void* x, int row_bytes, int T, const int32_t* topk_idx,
                            int top_k, int E, int32_t* offsets, int32_t* perm, int32_t* inv, void* xs, cudaStream_t s);
cudaError_t launch_combine(const TrainDevice& d, const void* ys, int dtype, int T, int H, int top_k, const int32_t* inv,
                           const float* w, void* out, cudaStream_t s);
cudaError_t launch_combine_backward(const TrainDevice& d, const void* dout, const void* ys, int dtype, int T, int H,
                                    int top_k, const int32_t* inv, const float* w, void* dys, float* dw,
                                    cudaStream_t s);
cudaError_t launch_route_backward(const TrainDevice& d, const float* logits, const int32_t* topk_idx,
                                  const float* topk_w, const float* dw, int T, int E, int top_k, int norm,
                                  float* dlogits, cudaStream_t s);

// Embedding (embed.cu).
struct EmbedWorkspace {
  int64_t keys[2], pos[2];  // byte offsets of the sort's two buffers of keys and positions
  int64_t part;             // [2 * chunks][H] fp32 sums of runs that leave their chunk
  int64_t bytes;
};
EmbedWorkspace embed_workspace(int64_t N, int H);
cudaError_t embed_set_limits(int* sort_ctas);
cudaError_t launch_embed(const TrainDevice& d, const void* table, int dtype, int64_t V, int H, const void* ids,
                         int id_bytes, int64_t N, float scale, void* out, cudaStream_t s);
cudaError_t launch_embed_backward(const TrainDevice& d, const void* dout, int dtype, const void* ids, int id_bytes,
                                  int64_t N, int64_t V, int H, float scale, int64_t padding_id, void* dtable,
                                  int table_dtype, bool accumulate, uint8_t* ws, cudaStream_t s);

// Policy loss (policy.cu).
cudaError_t policy_set_limits();
cudaError_t launch_policy_loss(const TrainDevice& d, const ftmoe_policy_args& a, cudaStream_t s);

// AdamW (adamw.cu).
cudaError_t launch_adamw(const TrainDevice& d, const ftmoe_adamw_tensor* list, int n, const ftmoe_adamw_params& hp,
                         cudaStream_t s);

}  // namespace ftmoe
