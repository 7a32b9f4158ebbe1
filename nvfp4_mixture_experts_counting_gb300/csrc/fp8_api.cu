// Entry points of the 8-bit layer: argument checks and launches.
#include <cmath>

#include "fp8.h"
#include "kernels.h"

using namespace ftmoe;

namespace {

constexpr int kMaxWidth = 1 << 24;

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return FTMOE_OK;
  cudaGetLastError();
  return cuda_fail(e, what);
}

bool on(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
bool known(int dtype) { return dtype == FTMOE_BF16 || dtype == FTMOE_FP32 || dtype == FTMOE_FP16; }
int bytes_of(int dtype) { return dtype == FTMOE_FP32 ? 4 : 2; }
bool width(int n) { return n > 0 && n <= kMaxWidth; }

int check_route(const ftmoe_route_args* a) {
  if (!a || !known(a->dtype) || a->T < 0 || a->E < 1 || a->E > kMaxBins || a->ld < a->E) return FTMOE_ERR_INVALID_ARG;
  if (a->score != FTMOE_SCORE_SOFTMAX && a->score != FTMOE_SCORE_SIGMOID) return FTMOE_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale) || a->scale == 0.f) return FTMOE_ERR_INVALID_ARG;
  if (a->n_groups < 1 || a->n_groups > kMaxGroups || a->E % a->n_groups) return FTMOE_ERR_INVALID_ARG;
  if (a->top_groups < 1 || a->top_groups > a->n_groups) return FTMOE_ERR_INVALID_ARG;
  if (a->group_best != 1 && a->group_best != 2) return FTMOE_ERR_INVALID_ARG;
  if (a->top_k < 1 || a->top_k > 32 || a->top_k > a->E / a->n_groups * a->top_groups) return FTMOE_ERR_INVALID_ARG;
  if (a->T > 0 && (!a->logits || !a->topk_idx || !a->topk_w)) return FTMOE_ERR_INVALID_ARG;
  if (!on(a->logits, bytes_of(a->dtype)) || !on(a->bias, 4) || !on(a->topk_idx, 4) || !on(a->topk_w, 4))
    return FTMOE_ERR_ALIGNMENT;
  return FTMOE_OK;
}

}  // namespace

extern "C" {

int ftmoe_route_topk(const ftmoe_route_args* args, ftmoe_stream_t stream) {
  if (const int rc = check_route(args)) return rc;
  if (args->T == 0) return FTMOE_OK;
  TrainDevice d;
  if (const int rc = train_device(&d)) return rc;
  return launched(launch_route_topk(d, *args, (cudaStream_t)stream), "ftmoe_route_topk");
}

int ftmoe_route_topk_backward(const ftmoe_route_args* args, const float* dw, void* dlogits, int64_t ld_d,
                              ftmoe_stream_t stream) {
  if (const int rc = check_route(args)) return rc;
  if (ld_d < args->E) return FTMOE_ERR_INVALID_ARG;
  if (args->T == 0) return FTMOE_OK;
  if (!dw || !dlogits || (dlogits == args->logits && ld_d != args->ld)) return FTMOE_ERR_INVALID_ARG;
  if (!on(dw, 4) || !on(dlogits, bytes_of(args->dtype))) return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = train_device(&d)) return rc;
  return launched(launch_route_topk_backward(d, *args, dw, dlogits, ld_d, (cudaStream_t)stream),
                  "ftmoe_route_topk_backward");
}

int ftmoe_fp8_quantize(const void* x, int dtype, int T, int K, const int32_t* inv, int top_k, const int32_t* used,
                       uint8_t* codes, float* scales, ftmoe_stream_t stream) {
  if (!known(dtype) || T < 0 || !width(K) || top_k < 1 || top_k > 32 || (!inv && top_k != 1) ||
      (int64_t)T * top_k > INT32_MAX)
    return FTMOE_ERR_INVALID_ARG;
  if (K % 16) return FTMOE_ERR_ALIGNMENT;
  if (T == 0) return FTMOE_OK;
  if (!x || !codes || !scales || x == codes) return FTMOE_ERR_INVALID_ARG;
  if (!on(x, 16) || !on(codes, 16) || !on(scales, 4) || !on(inv, 4) || !on(used, 4)) return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = train_device(&d)) return rc;
  return launched(launch_fp8_quantize(d, x, dtype, T, K, inv, top_k, used, codes, scales, (cudaStream_t)stream),
                  "ftmoe_fp8_quantize");
}

int ftmoe_fp8_quantize_weights(const void* w, int dtype, int E, int N, int K, uint8_t* codes, float* scales,
                               ftmoe_stream_t stream) {
  if (!known(dtype) || E < 0 || E > kMaxBins || !width(N) || !width(K)) return FTMOE_ERR_INVALID_ARG;
  if ((int64_t)fp8_blocks(N) * fp8_blocks(K) > INT32_MAX) return FTMOE_ERR_INVALID_ARG;
  if (K % 16) return FTMOE_ERR_ALIGNMENT;
  if (E == 0) return FTMOE_OK;
  if (!w || !codes || !scales || w == codes) return FTMOE_ERR_INVALID_ARG;
  if (!on(w, 16) || !on(codes, 16) || !on(scales, 4)) return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = train_device(&d)) return rc;
  return launched(launch_fp8_quantize_weights(d, w, dtype, E, N, K, codes, scales, (cudaStream_t)stream),
                  "ftmoe_fp8_quantize_weights");
}

int ftmoe_fp8_matmul(const ftmoe_fp8_matmul_args* a, ftmoe_stream_t stream) {
  if (!a || a->M < 0 || a->M > INT32_MAX || a->E < 1 || a->E > kMaxBins || !width(a->N) || !width(a->K))
    return FTMOE_ERR_INVALID_ARG;
  if ((!a->offsets && a->E != 1) || (a->transpose && a->swiglu)) return FTMOE_ERR_INVALID_ARG;
  if (!a->swiglu && !known(a->out_dtype)) return FTMOE_ERR_INVALID_ARG;
  // tiles of 128 rows and at least 128 columns are counted in 32 bits
  if ((a->M / 128 + a->E) * (((int64_t)(a->transpose ? a->K : a->N) + 127) / 128) > INT32_MAX) return FTMOE_ERR_INVALID_ARG;
  // a tensor map's strides are below 2^40 bytes
  if ((int64_t)a->N * a->K >= (int64_t)1 << 40) return FTMOE_ERR_INVALID_ARG;
  if (a->K % 16 || (a->transpose && a->N % 16) || (a->swiglu && a->N % (2 * kFp8Block))) return FTMOE_ERR_ALIGNMENT;
  if (a->M == 0) return FTMOE_OK;
  if (!a->a || !a->a_scale || !a->w || !a->w_scale || !a->out || a->out == a->a ||
      (a->swiglu && (!a->out_scale || a->out_scale == a->a_scale)))
    return FTMOE_ERR_INVALID_ARG;
  if (!on(a->a, 16) || !on(a->w, 16) || !on(a->out, 16) || !on(a->a_scale, 4) || !on(a->w_scale, 4) ||
      !on(a->offsets, 4) || !on(a->out_scale, 4))
    return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = train_device(&d)) return rc;
  return launched(launch_fp8_matmul(d, *a, (cudaStream_t)stream), "ftmoe_fp8_matmul");
}

static int swiglu_call(const void* gu, const void* dh, bool grad, int dtype, int rows, int I, const int32_t* used,
                       void* out, float* scales, cudaStream_t stream, const char* what) {
  if (!known(dtype) || rows < 0 || !width(I)) return FTMOE_ERR_INVALID_ARG;
  if (scales && I % kFp8Block) return FTMOE_ERR_ALIGNMENT;
  if (rows == 0) return FTMOE_OK;
  // a 16-bit gradient may take its input's place: a thread reads what it replaces
  if (!gu || !out || (grad && (!dh || out == dh)) || (out == gu && (!grad || scales))) return FTMOE_ERR_INVALID_ARG;
  if (!on(gu, 16) || !on(dh, 16) || !on(out, 16) || !on(scales, 4) || !on(used, 4)) return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = train_device(&d)) return rc;
  return launched(launch_swiglu(d, gu, dh, dtype, rows, I, used, out, scales, stream), what);
}

int ftmoe_swiglu(const void* gu, int dtype, int rows, int I, const int32_t* used, void* out, float* scales,
                 ftmoe_stream_t stream) {
  return swiglu_call(gu, nullptr, false, dtype, rows, I, used, out, scales, (cudaStream_t)stream, "ftmoe_swiglu");
}

int ftmoe_swiglu_backward(const void* dh, const void* gu, int dtype, int rows, int I, const int32_t* used, void* dgu,
                          float* scales, ftmoe_stream_t stream) {
  return swiglu_call(gu, dh, true, dtype, rows, I, used, dgu, scales, (cudaStream_t)stream, "ftmoe_swiglu_backward");
}

}  // extern "C"
