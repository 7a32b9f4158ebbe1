// Entry points of the training operators: argument checks, the current
// device's status word, and the launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <mutex>

#include "kernels.h"
#include "tma.cuh"
#include "train.h"

using namespace ftmoe;

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxH = 1 << 24;

static __device__ uint32_t g_ops_status[2];  // what the checks mark; what the latest reader took

std::mutex g_mu;
std::atomic<uint32_t> g_test_wait_ns{0};  // ftmoe_test_withhold_policy
std::mutex g_status_mu;  // one reader at a time: they share the second word
TrainDevice g_devices[kMaxDevices] = {};

// The word, cleared as it is read: a copy and a clearing apart would lose a
// mark that another stream makes between the two.
__global__ void k_take_status(uint32_t* status, uint32_t* taken) { *taken = atomicExch(status, 0u); }

// Once per device, with that device current: the status word's address and
// the kernels' shared-memory limits.
int current_device(TrainDevice* out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return FTMOE_ERR_DEVICE;
  }
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_devices[dev].status) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return FTMOE_ERR_DEVICE;
    }
    if (major != 10 || minor != 3) return FTMOE_ERR_DEVICE;
    void* p = nullptr;
    int sort_ctas = kSortCtas;
    cudaError_t e = cudaGetSymbolAddress(&p, g_ops_status);
    if (e == cudaSuccess) e = dispatch_set_limits(&sort_ctas);
    if (e == cudaSuccess) e = embed_set_limits(&sort_ctas);
    if (e == cudaSuccess) e = policy_set_limits();
    if (e != cudaSuccess) {
      cudaGetLastError();
      return cuda_fail(e, "training operators' set-up");
    }
    g_devices[dev] = {static_cast<uint32_t*>(p), sms, sort_ctas, 0};
  }
  *out = g_devices[dev];
  out->test_wait_ns = g_test_wait_ns;
  return FTMOE_OK;
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return FTMOE_OK;
  cudaGetLastError();
  return cuda_fail(e, what);
}

bool on(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
bool known(int dtype) { return dtype == FTMOE_BF16 || dtype == FTMOE_FP32 || dtype == FTMOE_FP16; }
int bytes_of(int dtype) { return dtype == FTMOE_FP32 ? 4 : 2; }

// Sizes that the expert-order calls share.
bool pair_sizes(int dtype, int T, int H, int top_k) {
  return known(dtype) && T >= 0 && H > 0 && H <= kMaxH && top_k > 0 && top_k <= 32 && (int64_t)T * top_k <= INT32_MAX;
}

}  // namespace

extern "C" {

int ftmoe_dispatch(const void* x, int dtype, int T, int H, const int32_t* topk_idx, int top_k, int E, int32_t* offsets,
                   int32_t* perm, int32_t* inv, void* xs, ftmoe_stream_t stream) {
  if (!pair_sizes(dtype, T, H, top_k) || E < 1 || E > kMaxBins || !offsets) return FTMOE_ERR_INVALID_ARG;
  if (T > 0 && (!topk_idx || !perm || !inv)) return FTMOE_ERR_INVALID_ARG;
  if ((!x) != (!xs) || (x && x == xs)) return FTMOE_ERR_INVALID_ARG;
  if (!on(x, 16) || !on(xs, 16) || !on(topk_idx, 4) || !on(offsets, 4) || !on(perm, 4) || !on(inv, 4))
    return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = current_device(&d)) return rc;
  return launched(launch_dispatch(d, x, H * bytes_of(dtype), T, topk_idx, top_k, E, offsets, perm, inv, xs,
                                  (cudaStream_t)stream),
                  "ftmoe_dispatch");
}

int ftmoe_combine(const void* ys, int dtype, int T, int H, int top_k, const int32_t* inv, const float* w, void* out,
                  ftmoe_stream_t stream) {
  if (!pair_sizes(dtype, T, H, top_k)) return FTMOE_ERR_INVALID_ARG;
  if (T == 0) return FTMOE_OK;
  if (!ys || !inv || !out || ys == out) return FTMOE_ERR_INVALID_ARG;
  if (!on(ys, 16) || !on(out, 16) || !on(inv, 4) || !on(w, 4)) return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = current_device(&d)) return rc;
  return launched(launch_combine(d, ys, dtype, T, H, top_k, inv, w, out, (cudaStream_t)stream), "ftmoe_combine");
}

int ftmoe_combine_backward(const void* dout, const void* ys, int dtype, int T, int H, int top_k, const int32_t* inv,
                           const float* w, void* dys, float* dw, ftmoe_stream_t stream) {
  if (!pair_sizes(dtype, T, H, top_k)) return FTMOE_ERR_INVALID_ARG;
  if (T == 0) return FTMOE_OK;
  if (!dout || !ys || !inv || !w || !dys || !dw || dys == dout) return FTMOE_ERR_INVALID_ARG;
  if (!on(dout, 16) || !on(ys, 16) || !on(dys, 16) || !on(inv, 4) || !on(w, 4) || !on(dw, 4))
    return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = current_device(&d)) return rc;
  return launched(launch_combine_backward(d, dout, ys, dtype, T, H, top_k, inv, w, dys, dw, (cudaStream_t)stream),
                  "ftmoe_combine_backward");
}

int ftmoe_route_backward(const float* logits, const int32_t* topk_idx, const float* topk_w, const float* dw, int T,
                         int E, int top_k, int norm_topk_prob, float* dlogits, ftmoe_stream_t stream) {
  if (T < 0 || E < 1 || E > kMaxBins || top_k < 1 || top_k > 32 || top_k > E) return FTMOE_ERR_INVALID_ARG;
  if (T == 0) return FTMOE_OK;
  if (!topk_idx || !topk_w || !dw || !dlogits || (!norm_topk_prob && !logits)) return FTMOE_ERR_INVALID_ARG;
  if (!on(logits, 4) || !on(topk_idx, 4) || !on(topk_w, 4) || !on(dw, 4) || !on(dlogits, 4))
    return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = current_device(&d)) return rc;
  return launched(launch_route_backward(d, logits, topk_idx, topk_w, dw, T, E, top_k, norm_topk_prob, dlogits,
                                        (cudaStream_t)stream),
                  "ftmoe_route_backward");
}

static bool embed_sizes(int dtype, int64_t V, int H, int id_bytes, int64_t N) {
  return known(dtype) && V >= 1 && V <= (1 << 30) && H > 0 && H <= kMaxH && (id_bytes == 4 || id_bytes == 8) &&
         N >= 0 && N <= INT32_MAX;
}

int ftmoe_embed(const void* table, int dtype, int64_t V, int H, const void* ids, int id_bytes, int64_t N, float scale,
                void* out, ftmoe_stream_t stream) {
  if (!embed_sizes(dtype, V, H, id_bytes, N)) return FTMOE_ERR_INVALID_ARG;
  if (N == 0) return FTMOE_OK;
  if (!table || !ids || !out || table == out) return FTMOE_ERR_INVALID_ARG;
  if (!on(table, 16) || !on(out, 16) || !on(ids, id_bytes)) return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = current_device(&d)) return rc;
  return launched(launch_embed(d, table, dtype, V, H, ids, id_bytes, N, scale, out, (cudaStream_t)stream),
                  "ftmoe_embed");
}

int64_t ftmoe_embed_workspace(int64_t N, int H) {
  if (N < 0 || N > INT32_MAX || H <= 0 || H > kMaxH) return FTMOE_ERR_INVALID_ARG;
  return embed_workspace(N, H).bytes;
}

int ftmoe_embed_backward(const void* dout, int dtype, const void* ids, int id_bytes, int64_t N, int64_t V, int H,
                         float scale, int64_t padding_id, void* dtable, int table_dtype, int accumulate,
                         void* workspace, int64_t workspace_bytes, ftmoe_stream_t stream) {
  if (!embed_sizes(dtype, V, H, id_bytes, N) || !known(table_dtype)) return FTMOE_ERR_INVALID_ARG;
  if (table_dtype != dtype && table_dtype != FTMOE_FP32) return FTMOE_ERR_INVALID_ARG;
  if (accumulate && table_dtype != FTMOE_FP32) return FTMOE_ERR_INVALID_ARG;
  if (!dtable || dtable == dout) return FTMOE_ERR_INVALID_ARG;
  if (N > 0 && (!dout || !ids || !workspace || workspace_bytes < embed_workspace(N, H).bytes))
    return FTMOE_ERR_INVALID_ARG;
  if (!on(dout, 16) || !on(dtable, 16) || !on(workspace, 16) || !on(ids, id_bytes)) return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = current_device(&d)) return rc;
  return launched(launch_embed_backward(d, dout, dtype, ids, id_bytes, N, V, H, scale, padding_id, dtable, table_dtype,
                                        accumulate != 0, static_cast<uint8_t*>(workspace), (cudaStream_t)stream),
                  "ftmoe_embed_backward");
}

int ftmoe_policy_loss(const ftmoe_policy_args* a, ftmoe_stream_t stream) {
  if (!a || !known(a->dtype) || (a->id_bytes != 4 && a->id_bytes != 8)) return FTMOE_ERR_INVALID_ARG;
  if (a->N < 0 || a->N > INT32_MAX || a->V < 1 || a->V > (1 << 30) || a->ld < a->V) return FTMOE_ERR_INVALID_ARG;
  if (!(a->temperature > 0.f) || !std::isfinite(a->temperature) || !(a->clip_low >= 0.f) || !(a->clip_high >= 0.f) ||
      !std::isfinite(a->kl_coef) || !std::isfinite(a->grad_scale))
    return FTMOE_ERR_INVALID_ARG;
  if (!a->loss) return FTMOE_ERR_INVALID_ARG;
  if (a->N > 0 && (!a->logits || !a->targets || !a->old_logp || !a->advantage || !a->row_loss))
    return FTMOE_ERR_INVALID_ARG;
  if (a->dlogits && a->ld_d < a->V) return FTMOE_ERR_INVALID_ARG;
  if (a->dlogits == a->logits && a->dlogits && a->ld_d != a->ld) return FTMOE_ERR_INVALID_ARG;
  const int b = bytes_of(a->dtype);
  if (!on(a->logits, b) || !on(a->dlogits, b) || !on(a->targets, a->id_bytes) || !on(a->old_logp, 4) ||
      !on(a->ref_logp, 4) || !on(a->advantage, 4) || !on(a->weight, 4) || !on(a->loss, 4) || !on(a->row_loss, 4) ||
      !on(a->logp, 4))
    return FTMOE_ERR_ALIGNMENT;
  TrainDevice d;
  if (const int rc = current_device(&d)) return rc;
  return launched(launch_policy_loss(d, *a, (cudaStream_t)stream), "ftmoe_policy_loss");
}

int ftmoe_test_withhold_policy(int enable, int64_t wait_limit_ns) {
  if (wait_limit_ns < 0 || wait_limit_ns > (int64_t)kWaitLimitNs) return FTMOE_ERR_INVALID_ARG;
  g_test_wait_ns = !enable ? 0 : wait_limit_ns ? (uint32_t)wait_limit_ns : (uint32_t)kWaitLimitNs;
  return FTMOE_OK;
}

int ftmoe_adamw(const ftmoe_adamw_tensor* tensors, int n, const ftmoe_adamw_params* hp, ftmoe_stream_t stream) {
  if (n < 0 || !hp || (n > 0 && !tensors)) return FTMOE_ERR_INVALID_ARG;
  if (!std::isfinite(hp->lr) || !(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0) ||
      !(hp->eps >= 0.0) || !std::isfinite(hp->eps) || hp->step < 1)
    return FTMOE_ERR_INVALID_ARG;
  if (!on(hp->grad_scale, 4)) return FTMOE_ERR_ALIGNMENT;
  bool any = false;
  for (int i = 0; i < n; ++i) {
    const ftmoe_adamw_tensor& t = tensors[i];
    if (t.n < 0 || !known(t.p_dtype) || !known(t.g_dtype) || (t.state_bits != 8 && t.state_bits != 32) ||
        !std::isfinite(t.weight_decay))
      return FTMOE_ERR_INVALID_ARG;
    if (t.g_dtype != t.p_dtype && t.g_dtype != FTMOE_FP32) return FTMOE_ERR_INVALID_ARG;
    if (t.master && t.p_dtype == FTMOE_FP32) return FTMOE_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    any = true;
    if (!t.p || !t.g || !t.m || !t.v || (t.state_bits == 8 && (!t.m_scale || !t.v_scale)))
      return FTMOE_ERR_INVALID_ARG;
    const int sb = t.state_bits / 8;
    if (!on(t.p, bytes_of(t.p_dtype)) || !on(t.g, bytes_of(t.g_dtype)) || !on(t.master, 4) || !on(t.m, sb) ||
        !on(t.v, sb) || !on(t.m_scale, 4) || !on(t.v_scale, 4))
      return FTMOE_ERR_ALIGNMENT;
  }
  if (!any) return FTMOE_OK;
  TrainDevice d;
  if (const int rc = current_device(&d)) return rc;
  return launched(launch_adamw(d, tensors, n, *hp, (cudaStream_t)stream), "ftmoe_adamw");
}

int ftmoe_ops_status(ftmoe_stream_t stream) {
  TrainDevice d;
  if (const int rc = current_device(&d)) return rc;
  const cudaStream_t s = (cudaStream_t)stream;
  uint32_t st = 0;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) {
    std::lock_guard<std::mutex> lk(g_status_mu);
    // on the stream itself: what it runs next marks a word that has been cleared
    k_take_status<<<1, 1, 0, s>>>(d.status, d.status + 1);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyAsync(&st, d.status + 1, 4, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) return launched(e, "ftmoe_ops_status");
  if (st & kStatusTimeout) return FTMOE_ERR_TIMEOUT;
  return st & kStatusRange ? FTMOE_ERR_DEVICE_CHECK : FTMOE_OK;
}

}  // extern "C"
