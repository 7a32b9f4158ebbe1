/*
 * ftmoe.h -- C ABI of libftmoe.so, a routed NVFP4 mixture-of-experts FFN layer
 * for one GB300 (sm_103a).
 *
 * The layer (pages, by title):
 *   [PR385] "feat(qwen4_exp): tensor parallelism for Qwen3.8-Flash-Next
 *           (offload backend)"
 *   [I62]   "Offloaded MoE ignores tensor parallelism: TP=2 is a regression,
 *           and the fix is not expert parallelism"
 *
 *   out_t = sum_j w_tj * Y_{t,j} + sigmoid(g . x_t) * S_t
 *
 * with a replicated router (softmax -> top-k, renormalised over the k chosen
 * when norm_topk_prob is set), NVFP4 expert banks (packed E2M1 codes, 16-wide
 * E4M3 scale blocks, per-row fp32 globals), SwiGLU experts whose gate_up is
 * [2I, H] (gate rows [0, I), up rows [I, 2I)) and down is [H, I], a bf16
 * shared expert, and the combine routed + sigmoid(gate) * shared formed
 * before any reduction ([PR385] "What this adds").  An intermediate window
 * [i0, i0 + I_loc) computes the partial sum that a rank owning that slice of
 * I would compute; partials over windows that cover I once add up to the
 * whole layer ([I62] "The fix that fits: TP-shard the offload banks").
 *
 * Numerics (the pages leave these open; the readings taken):
 *   - Activations are NVFP4 too: x per token and the SwiGLU output per pair
 *     are quantised in 16-blocks with E4M3 scale = RNE(amax / 6) and a global
 *     of 1.0, so each expert contraction is W4A4 with exact block products.
 *   - Top-k ties go to the lower expert index; slots are ordered by logit
 *     descending.  Indices are those of the exact logits: the kernel
 *     ranks fp32 logits, certifies the ranking with a rigorous error bound,
 *     and re-ranks uncertain candidates from compensated double-fp32 sums
 *     (about 2^-48 relative error).
 *   - Reductions are in a fixed order with no atomics on values, so results
 *     are bit-identical run to run ([PR385] "Correctness" traces run-to-run
 *     divergence to bf16 atomics in the expert kernels).
 *
 * Conventions for every entry point:
 *   - Return FTMOE_OK (0) or a negative ftmoe_status; nothing traps or aborts.
 *   - "device" pointers are CUDA device memory of the handle's device;
 *     "host" pointers are ordinary host memory.  All arrays are row-major and
 *     contiguous.  Device pointers must be 16-byte aligned.
 *   - ftmoe_stream_t is a cudaStream_t (NULL = the legacy default stream).
 *   - The caller owns x, out, the aux buffers and the stream; the library
 *     owns the banks and its workspace.
 */
#ifndef FTMOE_H_
#define FTMOE_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FTMOE_ABI_VERSION 3

typedef void* ftmoe_stream_t; /* a cudaStream_t */

typedef enum {
  FTMOE_OK = 0,
  FTMOE_ERR_INVALID_ARG = -1,      /* bad size, NULL pointer, T > max_tokens, ... */
  FTMOE_ERR_ALIGNMENT = -2,        /* i0 or I_loc not a multiple of 16, unaligned pointer */
  FTMOE_ERR_NOT_LOADED = -3,       /* forward on a layer whose bank was never loaded */
  FTMOE_ERR_SLICE_OUT_OF_RANGE = -4, /* forward window not inside the loaded window */
  FTMOE_ERR_OOM = -5,              /* a device or pinned allocation failed */
  FTMOE_ERR_CUDA = -6,             /* a CUDA runtime call failed (details: ftmoe_last_cuda_error) */
  FTMOE_ERR_TIMEOUT = -7,          /* a bounded device-side wait ran out */
  FTMOE_ERR_FAULT_INJECTED = -8,   /* FTMOE_FAULT selected this call to fail */
  FTMOE_ERR_DEVICE = -9,           /* no device, or not a compute capability 10.3 device */
  FTMOE_ERR_DEVICE_CHECK = -10,    /* an in-kernel range check failed (see ftmoe_check_status) */
  FTMOE_ERR_TOO_LARGE = -11        /* sizes exceed the fixed scratch of ftmoe_route_static */
} ftmoe_status;

/* out_flags of ftmoe_forward: the output type, optionally OR-ed with
 * ACCUMULATE and with ACT_BF16 */
enum {
  FTMOE_OUT_BF16 = 0,        /* out is bf16 [T, H] */
  FTMOE_OUT_FP32 = 1,        /* out is fp32 [T, H] */
  FTMOE_OUT_ACCUMULATE = 0x100, /* fp32 only: out += this window's partial, one rounding per add */
  FTMOE_ACT_BF16 = 0x200     /* W4A16 numerics: the routed experts take the bf16 x as it is and keep
                                their intermediate in bf16, weights dequantised in registers (the
                                weight-only 4-bit kernel the pages' review thread selects, [PR385]
                                mirror, kernel-selection fix); CUDA cores, meant for decode sizes;
                                resident mode only.  Default (flag clear): W4A4, activations NVFP4. */
};

typedef struct ftmoe_handle ftmoe_handle; /* opaque; library-owned */

typedef struct {
  int32_t abi_version;     /* = FTMOE_ABI_VERSION */
  int32_t H;               /* hidden size, multiple of 16 */
  int32_t I;               /* routed intermediate size, multiple of 16 */
  int32_t E;               /* routed experts, 1..1024 */
  int32_t top_k;           /* 1..min(E, 32) */
  int32_t I_shared;        /* shared-expert intermediate size, multiple of 16 (0 = no shared expert) */
  int32_t num_layers;      /* layers this handle holds banks for */
  int32_t max_tokens;      /* largest T a forward accepts; sizes the workspace once */
  int32_t norm_topk_prob;  /* 1: renormalise over the k chosen; 0: full-softmax probabilities */
  int32_t has_router_bias; /* 1: banks carry a per-expert router bias [E] */
  int64_t hbm_slot_bytes;  /* 0: all banks resident in HBM; > 0: offload mode.  The banks stay in
                              pinned host memory and the handle keeps
                              floor(hbm_slot_bytes / expert window bytes) expert slots in HBM,
                              shared by all layers, filled least-recently-used first (PR #385
                              "What this adds": a fraction of the experts resident, the rest
                              streamed every step).  Expert window bytes = 2*Iw*(H/2 + H/16 + 4)
                              + H*(Iw/2 + Iw/16 + 4) for the loaded window Iw; a slot physically
                              also holds the tensor-core copy of the scales (about 1/8 more). */
} ftmoe_config;

/* One layer's weights, as given to ftmoe_load_bank.  Every array is the full
 * (unsliced) tensor; the loader keeps only the window it is asked for.
 * Pointers are host memory when on_device == 0, else device memory. */
typedef struct {
  const float* router_w;       /* [E, H] fp32 */
  const float* router_bias;    /* [E] fp32, or NULL (required iff has_router_bias) */
  const uint8_t* gu_codes;     /* [E, 2I, H/2]  E2M1 pairs, element 2j in the low nibble */
  const uint8_t* gu_scales;    /* [E, 2I, H/16] E4M3 (fn) scale per 16-block */
  const float* gu_global;      /* [E, 2I]       fp32 per-row global */
  const uint8_t* dn_codes;     /* [E, H, I/2] */
  const uint8_t* dn_scales;    /* [E, H, I/16] */
  const float* dn_global;      /* [E, H] */
  const uint16_t* sh_gate_up;  /* [2*I_shared, H] bf16, gate rows first (NULL iff I_shared == 0) */
  const uint16_t* sh_down;     /* [H, I_shared] bf16 */
  const uint16_t* sh_gate;     /* [H] bf16 shared-expert gate vector */
  int32_t on_device;           /* 0 = host pointers, 1 = device pointers */
} ftmoe_bank_desc;

/* Optional outputs of ftmoe_forward (caller-owned device buffers; any may be NULL). */
typedef struct {
  int32_t* topk_idx;  /* [T, top_k] expert of each slot, slots by logit descending */
  float* topk_w;      /* [T, top_k] routing weight of each slot */
  int32_t* offsets;   /* [E + 1] first sorted position of each expert; offsets[E] = T*top_k */
  int32_t* perm;      /* [T*top_k] pair id p = t*top_k + j at each sorted position */
  int32_t* inv;       /* [T*top_k] sorted position of each pair id */
  float* logits;      /* [T, E] router logits (bias included) as the fast pass computed them,
                         before any re-rank of uncertain tokens */
  /* Each pair's quantised intermediate h = SiLU(G_gate) * G_up (NVFP4, global
     1.0, 16-blocks along the window), rows in sorted-position order:
     h_codes [T*top_k, I_loc/2] (two E2M1 codes a byte, low nibble first),
     h_scales [T*top_k, I_loc/16] (E4M3).  Written by ftmoe_forward's
     tensor-core prefill path only (resident banks, T > 32 and the shapes it
     takes); other paths and calls leave them untouched. */
  uint8_t* h_codes;
  uint8_t* h_scales;
} ftmoe_aux;

typedef struct {
  int32_t touched_experts;  /* distinct experts routed to by the last forward of this layer */
  int32_t resident_slots;   /* offload mode: HBM expert slots; resident mode: E */
  int64_t touched_bytes;    /* routed expert bytes the last forward read (window-restricted) */
  int64_t hits, misses;     /* offload mode: cumulative slot hits / misses of this layer */
  int64_t h2d_bytes;        /* offload mode: cumulative host->device expert bytes of this layer */
  double residency;         /* offload mode: resident slots / E; resident mode: 1.0 */
  int32_t device_status;    /* last device status word read by ftmoe_check_status */
  int64_t reranked_tokens;  /* cumulative tokens (all layers) whose top-k needed re-ranking */
  int64_t touched_total;    /* cumulative touched experts over every forward (all layers) */
} ftmoe_stats;

/* Create a handle on CUDA device `device` for layers of the given shape.
 * The shape is that of one MoE layer of the pages' model: E routed experts
 * with top_k chosen per token, gate_up [2I, H] and down [H, I] per expert,
 * a shared expert of intermediate I_shared gated by sigmoid(g . x)
 * ([PR385] "What this adds", first and third bullets; [I62] "What it
 * touches" for the [2I, H] / [H, I] shapes).  hbm_slot_bytes > 0 selects the
 * offload backend the pages are about: banks in pinned host memory and a
 * fraction of the experts resident in HBM slots ([PR385] "What this adds";
 * [I62] "Why TP=2 loses today").
 * Allocates the workspace for config->max_tokens (offload mode: also the
 * copy stream; the HBM slot pool follows at the first ftmoe_load_bank, once
 * the record size is known), so that a forward allocates nothing and, in
 * resident mode, can be captured in a CUDA graph ([I62] "The fix that
 * fits": "CUDA graphs unaffected. Shapes stay static").  Validates the config
 * (INVALID_ARG, ALIGNMENT) and the device (DEVICE).  On success *out owns
 * everything until ftmoe_destroy; on failure *out is NULL and nothing is
 * left allocated. */
int ftmoe_create(const ftmoe_config* config, int device, ftmoe_handle** out);

/* Load layer `layer`'s weights, keeping the intermediate window
 * [i0, i0 + I_loc) of every routed expert and of the shared expert: gate rows
 * [i0, i0+I_loc) and up rows [I+i0, I+i0+I_loc) of gate_up with their scales
 * and globals, and columns [i0, i0+I_loc) of down with their scale columns;
 * down keeps all H of its per-row globals ([I62] "What it touches": two
 * disjoint row ranges and a column slice; I/tp must stay a multiple of the
 * block size).  i0 and I_loc must be multiples of 16 (ALIGNMENT) and the
 * window inside [0, I) (INVALID_ARG).  The router and the shared gate vector
 * are loaded whole.  The call copies what it keeps (to HBM, or in offload mode
 * to pinned host memory) and synchronises `stream` before returning, so the
 * caller may free its buffers afterwards.  Loading a layer again replaces it. */
int ftmoe_load_bank(ftmoe_handle* h, int layer, const ftmoe_bank_desc* desc, int i0, int I_loc,
                    ftmoe_stream_t stream);

/* One forward of layer `layer` over T tokens (0 <= T <= max_tokens) for the
 * intermediate window [i0, i0 + I_loc), which must lie inside the loaded
 * window (SLICE_OUT_OF_RANGE) and be 16-aligned (ALIGNMENT).
 * It computes the partial output that a tensor-parallel rank owning that
 * window of every expert and of the shared expert would compute: the
 * replicated router, softmax and top-k (renormalised when norm_topk_prob is
 * set), the windowed gate_up rows, SwiGLU, the windowed down columns, and
 * routed + sigmoid(gate) * shared formed before any reduction ([PR385] "What
 * this adds", first to third bullets; [I62] "The fix that fits": the down
 * projection yields partial sums, and its first comment: norm_topk_prob and
 * a replicated router make the plain SUM of the partials exact).  The sums
 * run in a fixed order with no atomics on values, so a repeated call gives
 * the same bits ([PR385] "Correctness").
 *   x:   device, bf16 [T, H]
 *   out: device, [T, H] of the type out_flags names; must not alias x.
 *        With FTMOE_OUT_ACCUMULATE (fp32 only) the window's partial is added
 *        to out, so running the windows of a partition of I one after another
 *        into one buffer gives the full layer in a fixed order.
 *   aux: NULL or optional routing outputs (see ftmoe_aux).
 * Routing always uses the full replicated router.  Asynchronous on `stream`;
 * at prefill sizes the shared expert's products run on a stream of the
 * handle that waits for `stream`'s earlier work and that `stream` waits for
 * before the combine, so the call's work stays ordered within `stream`.
 * Resident mode does no host synchronisation and may be captured in a CUDA
 * graph (the capture follows the fork and the join).  Offload mode reads the step's routing back to the host once per
 * call (one synchronisation) to plan its slot copies; a forward touching more
 * experts than there are slots runs its experts in batches of at most the
 * slot count; offload needs the tensor-core shapes (H a multiple of 256,
 * windows multiples of 64 and at least 256 wide; INVALID_ARG otherwise) and
 * is not capturable.  T == 0 returns OK and does nothing. */
int ftmoe_forward(ftmoe_handle* h, int layer, const void* x, int T, void* out, int out_flags,
                  int i0, int I_loc, const ftmoe_aux* aux, ftmoe_stream_t stream);

/* Layers [0, num_layers) in sequence over T tokens, each on the previous
 * one's output renormalised by its RMS (x <- bf16(y / sqrt(mean(y^2) + 1e-6)),
 * no residual), as in a stack of MoE layers with nothing in between.
 *   x:   device bf16 [T, H] (read only)
 *   out: device bf16 [T, H], the last layer's output
 * Uses the whole loaded window of every layer.  Asynchronous; capturable in a
 * CUDA graph in resident mode. */
int ftmoe_forward_stack(ftmoe_handle* h, const void* x, int T, void* out, ftmoe_stream_t stream);

/* The renorm between the layers of ftmoe_forward_stack, on its own (the same
 * kernel): x[t] = bf16(y[t] / sqrt(mean_h(y[t][h]^2) + 1e-6)) for t < T,
 * sum of squares in fp32 (stack workload: "renormalised by RMS between
 * layers, with no attention").
 *   y: device fp32 [T, H];  x: device bf16 [T, H] (must not alias y)
 * Asynchronous on `stream`.  Returns FTMOE_ERR_INVALID_ARG for null pointers
 * or H, T < 0. */
int ftmoe_rms_renorm(const float* y, void* x, int T, int H, ftmoe_stream_t stream);

/* One rank's share of an expert-parallel layer: the routed slots of a
 * subset of the experts, plus optionally a window of the shared expert:
 *   out_t = sum over the slots j of token t whose expert is in the subset of
 *           w_tj * Y_(t,j)  +  sigmoid(g . x_t) * S_t over the shared window
 * (routing over all experts; shared_I_loc == 0 leaves the shared expert out).
 * expert_mask: host [E], nonzero for the experts of the subset.  Rank r of an
 * expert-parallel layer owns the experts e with e % world == r, the
 * alternative the pages weigh and reject for its all-to-all, its capture at
 * static shapes and its load imbalance under skewed routing ([I62] "Why not
 * expert parallelism proper"); giving rank r also window r of the shared
 * expert keeps the shared work evenly split, and the shares over a partition
 * of the experts and of the shared window add up to the whole layer.  It
 * exists to measure that alternative against the intermediate split on the
 * same GPU.  The routed experts use the whole loaded window; the shared
 * window [shared_i0, shared_i0 + shared_I_loc) must lie in the loaded shared
 * window (SLICE_OUT_OF_RANGE) and be 16-aligned (ALIGNMENT).  Reads the
 * routing back to the host once (one synchronisation); resident mode only;
 * T <= 32 on the tensor-core decode shapes and T > 32 on the prefill shapes
 * (INVALID_ARG otherwise). */
int ftmoe_forward_experts(ftmoe_handle* h, int layer, const void* x, int T, void* out, int out_flags,
                          const uint8_t* expert_mask, int shared_i0, int shared_I_loc, const ftmoe_aux* aux,
                          ftmoe_stream_t stream);

/* The combine of an intermediate-sharded layer: each of n_parts ranks (or
 * windows) computed its fp32 partial of the same T tokens (ftmoe_forward
 * with FTMOE_OUT_FP32 on its window), the partials were exchanged into one
 * device buffer parts [n_parts][n] in rank order (n = T * H), and this sums
 * every element over the ranks in rank order and rounds it once to the
 * output type of out_flags (FTMOE_OUT_BF16, FTMOE_OUT_FP32, optionally
 * FTMOE_OUT_ACCUMULATE).  The pages' TP patch combines the ranks' partials
 * of routed + sigmoid(gate) * shared with one SUM per MoE layer ([PR385]
 * "What this adds", third bullet; [I62] "The fix that fits": "No new
 * collectives"); a fixed rank order keeps that sum identical run to run
 * ([PR385] "Correctness").  parts must be 16-byte aligned.  Asynchronous. */
int ftmoe_reduce_partials(const float* parts, int n_parts, int64_t n, void* out, int out_flags,
                          ftmoe_stream_t stream);

/* Release everything the handle owns (device workspace, banks, pinned host
 * banks and HBM slots of the offload backend, its copy stream).  Safe on
 * NULL.  Synchronises nothing: the caller makes sure no forward of this
 * handle is still running on its streams. */
int ftmoe_destroy(ftmoe_handle* h);

/* Static description of a status code. */
const char* ftmoe_error_string(int code);

/* Text of the last CUDA error seen by this thread's calls ("" if none). */
const char* ftmoe_last_cuda_error(void);

/* Per-layer counters (see ftmoe_stats): the touched experts and bytes of the
 * last forward, and, for the offload backend, the slot residency, hits,
 * misses and host-to-device bytes the pages measure the backend by ([PR385]
 * "Measurements": residency and cache slots; [I62] "Why TP=2 loses today":
 * slot counts per rank).  The routing-dependent fields are read back from
 * the device, so this call synchronises the handle's device. */
int ftmoe_get_stats(ftmoe_handle* h, int layer, ftmoe_stats* out);

/* Synchronise `stream`, read the device status word that the kernels set on a
 * failed range check or an expired bounded wait, clear it, and return OK,
 * DEVICE_CHECK or TIMEOUT.  After TIMEOUT the handle's cross-CTA counters
 * are cleared too, so the next forward starts clean.  The pages have no
 * counterpart; it is how a failure inside a kernel reaches the caller
 * without trapping the GPU. */
int ftmoe_check_status(ftmoe_handle* h, ftmoe_stream_t stream);

/* Test hook of the device-side failure path, off by default; the pages have
 * no counterpart.  While enabled (enable = 1), one CTA of every forward's
 * tensor-core decode down kernel never issues its first pipeline stage, so
 * its bounded waits give up after wait_limit_ns (0: the default limit of one
 * second): the kernel sets the status word's timeout bit, drains its copies,
 * frees its tensor memory and returns, and its output tile is not written.
 * ftmoe_check_status then returns FTMOE_ERR_TIMEOUT.  No GPU fault or trap
 * is involved.  INVALID_ARG if the handle has no tensor-core decode path. */
int ftmoe_test_withhold_stage(ftmoe_handle* h, int enable, int64_t wait_limit_ns);

/* Per-kernel timing.  While enabled, every kernel the handle launches is
 * bracketed by two CUDA events recorded on its launch stream.  Reading
 * synchronises those events, returns one entry per kernel name (launches,
 * summed event time in ms) in first-launch order, and clears the record.
 * Recording stays off by default; the events cost a few microseconds of host
 * time per launch.  n_out receives the number of entries (<= max_entries). */
typedef struct {
  char name[48];
  int64_t launches;
  double total_ms;
} ftmoe_kernel_time;

int ftmoe_profile_enable(ftmoe_handle* h, int enable);
int ftmoe_profile_read(ftmoe_handle* h, ftmoe_kernel_time* out, int max_entries, int* n_out);

/* NVFP4-quantise fp32 weight rows on the device (a load-time tool; the same
 * block arithmetic the forward applies to activations):
 *   g = fp32(row_amax / 2688); per 16-block s = E4M3(fp32(fp32(amax / 6) / g));
 *   code = E2M1(fp32(w / fp32(dec(s) * g))), round-to-nearest-even and
 *   saturating; zero rows, zero scales and zero denominators give zero codes.
 *   w:       device fp32 [rows, K], K a multiple of 16
 *   codes:   device [rows, K/2]; scales: device [rows, K/16]; globals: device fp32 [rows]
 * Asynchronous on `stream`. */
int ftmoe_quantize_weights(const float* w, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                           float* globals, ftmoe_stream_t stream);

/* Routing that allocates nothing.  The pages have no counterpart to this
 * entry point; it exists for callers that cannot call cudaMalloc when they
 * route: a serving runtime that has given all free device memory to its KV
 * cache and graph pools up front, a host that forbids device allocations
 * from plugins, or code running while a CUDA graph is captured.
 *
 * It runs the same router, top-k and counting-sort kernels as ftmoe_forward
 * and returns what ftmoe_forward's aux outputs return, with no handle.  All
 * pointers are device memory of the current device:
 *   x:        bf16 [T, H] (16-byte aligned), H a multiple of 16
 *   router_w: fp32 [E, H] (16-byte aligned); router_bias: fp32 [E] or NULL
 *   topk_idx [T, top_k], topk_w [T, top_k], offsets [E + 1],
 *   perm [T*top_k], inv [T*top_k]: outputs, as in ftmoe_aux.
 * Its scratch is one fixed array in the library's device image (287 KB per
 * device that loads the library, held until the process exits),
 * which bounds the sizes: T <= 1024, E <= 1024, T*E <= 16384,
 * T*H <= 262144 and H <= 8192; larger problems return FTMOE_ERR_TOO_LARGE.
 * The first call on a device looks up that array's device address (and sets
 * the kernels' shared-memory limits); make that first call before any stream
 * capture.  Every call shares the one array, so calls whose kernels overlap
 * on the GPU (different streams, or several threads) race: serialise them.
 * Asynchronous on `stream`; calls no allocating routine. */
int ftmoe_route_static(const void* x, int T, int H, const float* router_w, const float* router_bias, int E,
                       int top_k, int norm_topk_prob, int32_t* topk_idx, float* topk_w, int32_t* offsets,
                       int32_t* perm, int32_t* inv, ftmoe_stream_t stream);

/* Device-side checks of the latest ftmoe_route_static call on the current
 * device (the kernels' range checks: an expert index out of range is routed
 * to expert 0 and marked here).  Synchronises `stream`, reads and clears the
 * status word kept in the same fixed array, and returns OK, DEVICE_CHECK or
 * TIMEOUT.  Allocates nothing.  The pages have no counterpart. */
int ftmoe_route_static_status(ftmoe_stream_t stream);

/* Bank formats that ftmoe_slice_format slices (the pages' loader handles
 * several; [I62] "What it touches" and "Suggested staging").  Per expert, a
 * matrix W [N, K] (gate_up: N = 2I, K = H; down: N = H, K = I) is held as:
 *   NVFP4      arrays {codes [N][K/2], E4M3 scales [N][K/16], fp32 globals [N]}
 *   FP8_BLOCK  arrays {E4M3 q [N][K], fp32 scale [ceil(N/128)][ceil(K/128)]},
 *              W[n][k] = q[n][k] * scale[n/128][k/128]
 *   Q4_0       array  {blocks [N][K/32][18]}: fp16 scale d, then 16 bytes of
 *              4-bit codes (byte j: element j low nibble, j+16 high nibble),
 *              value = d * (code - 8)
 *   MXFP4      arrays {blocks_t [K/2][N], UE8M0 scales_t [K/32][N]}: stored
 *              transposed, byte [j][n] holds elements (n, 2j) low and
 *              (n, 2j+1) high, value = e2m1 * 2^(scale - 127) */
typedef enum {
  FTMOE_FMT_NVFP4 = 0,
  FTMOE_FMT_FP8_BLOCK = 1,
  FTMOE_FMT_Q4_0 = 2,
  FTMOE_FMT_MXFP4 = 3
} ftmoe_format;

enum { FTMOE_MAT_GATE_UP = 0, FTMOE_MAT_DOWN = 1 };

/* Slice E experts' gate_up or down matrix, held in `format`, to the
 * intermediate window [i0, i0 + I_loc) ([I62] "What it touches": gate_up
 * keeps two disjoint row ranges, gate rows [i0, i0+I_loc) then up rows
 * [I+i0, I+i0+I_loc); down keeps the columns [i0, i0+I_loc); mxfp4, stored
 * transposed, slices gate_up along its columns and down along its rows; the
 * NVFP4 down row globals stay whole).  src[i] / dst[i] are device pointers
 * to the format's arrays in the order listed above, for all E experts back
 * to back; the sliced arrays have the same layout at I_loc in place of I
 * (fp8_block: whole 128-row scale tiles of each part).  i0, I_loc, I and H
 * must be multiples of the format's block size (16 NVFP4, 128 FP8_BLOCK,
 * 32 Q4_0 and MXFP4: [I62] "Divisibility"), else FTMOE_ERR_ALIGNMENT; a
 * window outside [0, I) is FTMOE_ERR_INVALID_ARG.  Asynchronous on
 * `stream`; a load-time step, not part of the forward. */
int ftmoe_slice_format(int format, int matrix, int E, int H, int I, int i0, int I_loc, const void* const* src,
                       void* const* dst, ftmoe_stream_t stream);

/* NVFP4-quantise bf16 activation rows with the global fixed at 1.0 (the
 * forward's own activation quantiser, exposed for testing):
 *   a: device bf16 [rows, K]; codes [rows, K/2]; scales [rows, K/16]. */
int ftmoe_quantize_activations(const void* a, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                               ftmoe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Training operators: what one training step needs around the layer's matrix
 * products.  The pages serve the layer and have no counterpart.
 *
 * They need no handle: the caller owns every buffer, and the calls run on the
 * current device.  All are asynchronous on `stream`, allocate nothing, read
 * nothing back to the host and may be captured in a CUDA graph once one of
 * them has run on the device (the first call looks up a device address and
 * sets kernel limits).  Sums run in fp32 or wider in a fixed order and are
 * rounded once, so results are bit-identical run to run (onto an existing
 * table the embedding gradient adds once to each value, as a reduction).  Any
 * H, T, k and E within the limits below is taken; rows whose bytes are a
 * multiple of 16 move 16 bytes at a time.
 *
 * Range checks inside the kernels (an expert, place, id or target out of
 * range) mark a device word and leave the item out, as each call says;
 * ftmoe_ops_status reads that word. */
typedef enum { FTMOE_BF16 = 0, FTMOE_FP32 = 1, FTMOE_FP16 = 2 } ftmoe_dtype;

/* Sort the tokens' rows by expert.  Pair p = t*top_k + j has expert
 * topk_idx[t][j]; a negative expert drops the pair (a slot that another rank
 * owns), and so does one >= E, which also marks the status word.
 *   x:        [T, H] of `dtype`, or NULL (tables only)
 *   topk_idx: int32 [T, top_k], top_k 1..32, E 1..1024
 *   offsets:  [E + 1] first place of each expert; offsets[E] = pairs kept
 *   perm:     [T*top_k] pair at each place, by expert and then by pair id;
 *             -1 from offsets[E] on
 *   inv:      [T*top_k] place of each pair, -1 if it is dropped
 *   xs:       [T*top_k, H]: xs[inv[p]] = x[t]; rows from offsets[E] on stay
 *             as they were.  NULL iff x is.
 * offsets, perm and inv have ftmoe_aux's meaning when nothing is dropped.
 * The gradient of the copy is ftmoe_combine without weights.  T == 0 writes
 * offsets.  x and xs: 16-byte aligned, not the same. */
int ftmoe_dispatch(const void* x, int dtype, int T, int H, const int32_t* topk_idx, int top_k, int E,
                   int32_t* offsets, int32_t* perm, int32_t* inv, void* xs, ftmoe_stream_t stream);

/* out[t] = sum_j w[t][j] * ys[inv[t*top_k + j]] over the kept slots, in slot
 * order; a token without one gets zeros.  w: fp32 [T, top_k], or NULL for
 * weights of one.  A place outside [-1, T*top_k) counts as dropped and marks
 * the status word.  ys: [T*top_k, H], whose rows of no pair may hold anything;
 * ys, out: `dtype`, 16-byte aligned, not the same. */
int ftmoe_combine(const void* ys, int dtype, int T, int H, int top_k, const int32_t* inv, const float* w, void* out,
                  ftmoe_stream_t stream);

/* ftmoe_combine's gradient: dys[inv[p]] = w[p] * dout[t] (rows that no kept
 * pair has stay as they were) and dw[p] = <dout[t], ys[inv[p]]>, 0 for a
 * dropped pair.  ys and dys: [T*top_k, H]; dys may be ys itself (the rows are
 * replaced).  Places out of range as for ftmoe_combine. */
int ftmoe_combine_backward(const void* dout, const void* ys, int dtype, int T, int H, int top_k, const int32_t* inv,
                           const float* w, void* dys, float* dw, ftmoe_stream_t stream);

/* The router's gradient from that of its weights.  With S = sum_j w_j dw_j:
 *   norm_topk_prob: dlogits[e] = sum over the j with idx_j = e of w_j (dw_j - S)
 *                   (logits is not read and may be NULL)
 *   otherwise:      dlogits[e] = p_e (sum over those j of dw_j - S),
 *                   p = softmax(logits), logits fp32 [T, E] with the bias
 * topk_idx is the router's own choice, before any slot is dropped; an index
 * outside [0, E) is left out and marks the status word.  dlogits: fp32
 * [T, E], written whole; may be `logits` itself.  For ftmoe_route_static's
 * router; that of ftmoe_route_topk has ftmoe_route_topk_backward, which also
 * takes 16-bit logits, sigmoid scores, a scale, masked logits and slots of -1. */
int ftmoe_route_backward(const float* logits, const int32_t* topk_idx, const float* topk_w, const float* dw, int T,
                         int E, int top_k, int norm_topk_prob, float* dlogits, ftmoe_stream_t stream);

/* out[n] = scale * table[ids[n]].  ids: int32 or int64 (id_bytes 4 or 8); an
 * id outside [0, V) gives a row of zeros and marks the status word.
 * table [V, H], out [N, H]: `dtype`, 16-byte aligned, not the same. */
int ftmoe_embed(const void* table, int dtype, int64_t V, int H, const void* ids, int id_bytes, int64_t N, float scale,
                void* out, ftmoe_stream_t stream);

/* Bytes of the workspace that ftmoe_embed_backward needs for N tokens of
 * width H (about 16 N + N H / 4; negative: a status code). */
int64_t ftmoe_embed_workspace(int64_t N, int H);

/* ftmoe_embed's gradient: dtable[v] = scale * (sum over the n with ids[n] = v
 * of dout[n], in fp32).  The order of that sum is fixed: the tokens by id and
 * n in chunks of 32, each summed in the order of n, then an id's chunks in
 * order (over 16 of them: every eighth together, then those eight sums).
 * Rows of no token become zeros;
 * with `accumulate` (fp32 dtable only) the sum is added to dtable, where values
 * below the smallest normal one may count as zero, and other rows are not
 * touched.  Tokens whose id is padding_id are left out (-1: none
 * of the valid ids); other ids outside [0, V) are left out and mark the
 * status word.  V up to 2^30.
 *   dout: `dtype` [N, H]; dtable: table_dtype (`dtype` or FTMOE_FP32) [V, H]
 *   workspace: workspace_bytes >= ftmoe_embed_workspace(N, H); its contents
 *   matter only during the call */
int ftmoe_embed_backward(const void* dout, int dtype, const void* ids, int id_bytes, int64_t N, int64_t V, int H,
                         float scale, int64_t padding_id, void* dtable, int table_dtype, int accumulate,
                         void* workspace, int64_t workspace_bytes, ftmoe_stream_t stream);

/* Clipped policy loss with a KL term, and its gradient.  For each row n, with
 * z = logits[n] / temperature and y = targets[n]:
 *   logp = z_y - log(sum_v exp z_v),  r = exp(logp - old_logp),  A = advantage
 *   row  = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *          + kl_coef (exp(d) - d - 1),  d = ref_logp - logp
 *   loss = sum_n weight_n row_n
 *   dlogits[n] = grad_scale * weight_n * d row / d logits[n]
 * (the clipped side has no gradient; where both sides are equal the unclipped
 * one's is taken).  A row of weight 0 is left out: its logits are not read,
 * row_loss and logp are 0 and its gradient is zeros.  So is a row whose target
 * is outside [0, V), which also marks the status word.  Logits of -inf have
 * probability 0; NaN in a counted row reaches its outputs. */
typedef struct {
  const void* logits;      /* [N, V] of `dtype`, rows `ld` values apart (ld >= V); any row alignment */
  int32_t dtype;
  int32_t id_bytes;        /* 4 or 8: the targets' type */
  int64_t N, V, ld;
  const void* targets;     /* int32 or int64 [N] */
  const float* old_logp;   /* [N] log probability under the policy that sampled */
  const float* ref_logp;   /* [N] under the reference policy, or NULL (no KL term) */
  const float* advantage;  /* [N] */
  const float* weight;     /* [N], e.g. mask / number of counted tokens; NULL: 1/N each */
  float temperature;       /* > 0 */
  float clip_low, clip_high; /* >= 0 */
  float kl_coef;           /* 0: no KL term */
  float grad_scale;        /* of the gradient only (loss scaling) */
  float* loss;             /* [1] */
  float* row_loss;         /* [N], before the weight */
  float* logp;             /* [N] or NULL */
  void* dlogits;           /* [N, V] of `dtype`, rows ld_d apart, or NULL (forward only);
                              may be `logits` itself with ld_d == ld */
  int64_t ld_d;
} ftmoe_policy_args;

int ftmoe_policy_loss(const ftmoe_policy_args* args, ftmoe_stream_t stream);

/* Test hook of ftmoe_policy_loss's failure path, off by default and shared by
 * all threads.  While enabled, one warp of a call's first row never asks for
 * its first chunk of it, and the call's waits give up after wait_limit_ns (0:
 * the default limit of one second, which is the most).  The kernel sets the
 * status word's timeout bit and finishes: that row and those that the same
 * warp takes part in later come out as NaN, others as usual.  Rows that no
 * cluster's shared memory holds are not waited for.  No GPU fault or trap is
 * involved. */
int ftmoe_test_withhold_policy(int enable, int64_t wait_limit_ns);

/* One AdamW step over n_tensors tensors.  With g' = grad_scale * g and `step`
 * counted from 1:
 *   m <- beta1 m + (1 - beta1) g';  v <- beta2 v + (1 - beta2) g'^2
 *   p <- p (1 - lr weight_decay)
 *        - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in fp32.  Tensors may differ in size, types and weight decay; pointers need
 * only their own type's alignment.  With `master`, p is its rounded copy.
 * state_bits 8: m and v hold one E4M3 code a value, v's of the root sqrt(v),
 * with a scale per 256 consecutive values, scale = amax * fl(1/448) and code =
 * E4M3(value * (448 * fl(1/amax))) in fp32 (blocks whose amax is below 1e-30
 * are held as zeros); a root above zero keeps at least the smallest code.
 * Codes are rounded to nearest in 3 bits, so a root stays where a step changes
 * it by less than 3 to 6 %: against the exact one it settles at 1.06 times
 * (0.92 to 1.24 in nine of ten values) with beta2 = 0.95, 1.36 (1.12 to 1.66)
 * with 0.99 and 1.10 (0.71 to 1.49) with 0.999, for gradients of one size in a
 * block.  States of 32 bits have no such offset.
 * Zeros in codes and scales are the state before the first step.  A gradient
 * of NaN spoils its own value.  So does an infinite one, which in 8 bits also
 * makes the block's scales infinite: the next step spoils the whole block. */
typedef struct {
  void* p;               /* [n] of p_dtype, updated */
  const void* g;         /* [n] of g_dtype */
  float* master;         /* [n] fp32, updated, or NULL (p itself is the master); 16-bit p only */
  void* m;               /* [n] fp32, or uint8 codes */
  void* v;               /* [n] fp32, or uint8 codes of sqrt(v) */
  float* m_scale;        /* [ceil(n / 256)], 8-bit states only */
  float* v_scale;
  int64_t n;
  float weight_decay;
  int32_t p_dtype;
  int32_t g_dtype;       /* p_dtype or FTMOE_FP32 */
  int32_t state_bits;    /* 8 or 32 */
} ftmoe_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps;
  int64_t step;
  const float* grad_scale; /* device [1] or NULL (1); not finite: the whole step is skipped */
} ftmoe_adamw_params;

/* `tensors` and `params` are host memory, read during the call (the launches
 * carry the list: no device copy of it is made). */
int ftmoe_adamw(const ftmoe_adamw_tensor* tensors, int n_tensors, const ftmoe_adamw_params* params,
                ftmoe_stream_t stream);

/* ---------------------------------------------------------------------------
 * The layer on banks of 8-bit codes: routing from logits, the quantiser, the
 * experts' products and SwiGLU, with the gradients that pass through them to
 * the tokens and the router.  The pages serve their banks through formats
 * that this product reads one of (FTMOE_FMT_FP8_BLOCK) and have no
 * counterpart to the calls.
 *
 * Like the training operators they need no handle, run on the current device,
 * are asynchronous on `stream`, allocate nothing, may be captured once one of
 * them has run on the device, give the same bits run to run, and mark the word
 * that ftmoe_ops_status reads.  Matrices are dense and their pointers 16-byte
 * aligned, but for the router's logits.  One forward pass of a layer:
 *
 *   ftmoe_route_topk       logits -> experts and weights of each token
 *   ftmoe_dispatch         (x NULL) tables of the pairs sorted by expert
 *   ftmoe_fp8_quantize     tokens -> codes in their experts' rows
 *   ftmoe_fp8_matmul       gate_up with SwiGLU -> codes of the intermediate
 *   ftmoe_fp8_matmul       down -> rows
 *   ftmoe_combine          rows -> tokens
 *
 * and to train through it (codes are not trained: the bank stays as it is)
 * gate_up without `swiglu`, ftmoe_swiglu; then back ftmoe_combine_backward,
 * ftmoe_fp8_quantize (inv NULL), ftmoe_fp8_matmul with `transpose`,
 * ftmoe_swiglu_backward, ftmoe_fp8_matmul with `transpose`, ftmoe_combine
 * without weights, and ftmoe_route_topk_backward.
 *
 * Codes are E4M3 (fn) bytes.  Activations have a scale for 128 consecutive
 * values of a row, stored block by block: scales [ceil(K/128)][rows].  A block
 * of largest magnitude a has scale = fl(a / 448) and code = E4M3(x fl(448 / a))
 * in fp32, round to nearest even; blocks with a < 1e-30 are held as zeros; a
 * NaN or an infinity spoils its block.  Weights are FTMOE_FMT_FP8_BLOCK's
 * arrays: codes [E][N][K], scales [E][ceil(N/128)][ceil(K/128)]. */

typedef enum { FTMOE_SCORE_SOFTMAX = 0, FTMOE_SCORE_SIGMOID = 1 } ftmoe_score;

/* Experts of each token.  With l = logits[t]:
 *   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),  c_e = s_e + bias_e
 *   the E experts are n_groups equal groups in order; a group is worth the sum
 *   of its group_best largest c (of one, if only one is available), and only
 *   the experts of the top_groups best groups stay
 *   slots 0..top_k-1: the largest c among them, largest first
 *   w_j = scale s_j / (sum of s over the chosen), or scale s_j without
 *   norm_topk_prob
 * Ties go to the lower group and the lower expert.  Experts are ranked by their
 * logits where these decide (no bias, and one group or group_best 1), else as by
 * fp64 arithmetic on the given logits and biases.  An expert whose logit or
 * bias is -inf is not available, nor is one whose logit is NaN or +inf or whose
 * bias is not finite, which also marks the status word.  Slots that no expert
 * is left for get index -1 and weight 0 (ftmoe_dispatch drops them). */
typedef struct {
  const void* logits;     /* [T, E] of `dtype`, rows `ld` values apart (ld >= E), any alignment */
  int32_t dtype;          /* ftmoe_dtype */
  int32_t T, E;           /* E 1..1024 */
  int64_t ld;
  int32_t score;          /* ftmoe_score */
  int32_t top_k;          /* 1..32, at most top_groups * E / n_groups */
  int32_t norm_topk_prob;
  float scale;            /* of the weights; not 0 */
  const float* bias;      /* [E] or NULL: for the choice only (balance) */
  int32_t n_groups;       /* 1..32, a divisor of E */
  int32_t top_groups;     /* 1..n_groups */
  int32_t group_best;     /* 1 or 2 */
  int32_t* topk_idx;      /* [T, top_k] */
  float* topk_w;          /* [T, top_k] */
} ftmoe_route_args;

int ftmoe_route_topk(const ftmoe_route_args* args, ftmoe_stream_t stream);

/* Its gradient: dlogits [T, E] of `dtype`, rows ld_d apart, from dw [T, top_k],
 * the gradient of topk_w; topk_idx and topk_w are the forward call's.  The
 * choice itself and the bias have none.  Written whole; slots of -1 have no
 * part, an index outside [-1, E) is left out and marks the status word, equal
 * indices add up.  dlogits may be logits itself (ld_d == ld).
 * (ftmoe_route_backward is ftmoe_route_static's: there -1 marks the status word
 * too, and every logit counts.) */
int ftmoe_route_topk_backward(const ftmoe_route_args* args, const float* dw, void* dlogits, int64_t ld_d,
                              ftmoe_stream_t stream);

/* Quantise T rows of x [T, K] of `dtype`, K a multiple of 16.  Without inv
 * (top_k 1) row t goes to row t of codes [T, K] and scales [ceil(K/128)][T].
 * With inv [T * top_k] (ftmoe_dispatch's) it goes to the rows inv[t*top_k + j]
 * of codes [T*top_k, K] and scales [ceil(K/128)][T*top_k]; -1 drops a pair, a
 * place out of range drops it and marks the status word, and rows of no pair
 * stay as they were.  `used`: NULL, or the device count of rows of x to handle
 * (e.g. offsets + E), held to [0, T] with a mark. */
int ftmoe_fp8_quantize(const void* x, int dtype, int T, int K, const int32_t* inv, int top_k, const int32_t* used,
                       uint8_t* codes, float* scales, ftmoe_stream_t stream);

/* Quantise E matrices w [E][N][K] of `dtype` to FTMOE_FMT_FP8_BLOCK's arrays,
 * K a multiple of 16 (a load-time tool). */
int ftmoe_fp8_quantize_weights(const void* w, int dtype, int E, int N, int K, uint8_t* codes, float* scales,
                               ftmoe_stream_t stream);

/* Rows of each expert times its matrix.  Rows offsets[e] .. offsets[e+1] - 1
 * belong to expert e:
 *   out[r][n] = sum_k x[r][k] w[e][n][k]                      a [M, K], out [M, N]
 *   transpose:  out[r][k] = sum_n x[r][n] w[e][n][k]          a [M, N], out [M, K]
 *   swiglu:     h[r][i] = SwiGLU(y[r][i], y[r][N/2 + i]) of the first form's y,
 *               quantised: out codes [M, N/2], out_scale [N/256][M]
 * x and w are the values that codes and scales stand for.  Products are exact,
 * summed on the tensor cores over a block of 128 and in fp32 over the blocks.
 * The scales of a block, the rows' and the weights', are multiplied in fp32
 * first: where that product is below 2^-126 the block loses bits or vanishes,
 * and from 2^128 on it comes out infinite or NaN.  y is not rounded before
 * SwiGLU; there SiLU of y is within (1.25 |y| + 8) 2^-24 of itself, and 0 below
 * -87.3, before h's rounding to a code.  Rows of no expert (from offsets[E] on) stay
 * as they were and may hold anything.  An expert whose rows begin before an
 * earlier one's first row, fall or leave [0, M] is left out and marks the
 * status word. */
typedef struct {
  const uint8_t* a;        /* codes of the rows */
  const float* a_scale;    /* [ceil(K/128)][M]; transpose: [ceil(N/128)][M] */
  const uint8_t* w;        /* [E][N][K] */
  const float* w_scale;    /* [E][ceil(N/128)][ceil(K/128)] */
  const int32_t* offsets;  /* device [E + 1], or NULL with E == 1: all M rows */
  int64_t M;
  int32_t E, N, K;         /* N K < 2^40; K a multiple of 16; transpose: N too; swiglu: N a multiple of 256 */
  int32_t transpose, swiglu;
  int32_t out_dtype;       /* ftmoe_dtype (not with swiglu) */
  void* out;               /* not a */
  float* out_scale;        /* swiglu only; not a_scale */
} ftmoe_fp8_matmul_args;

int ftmoe_fp8_matmul(const ftmoe_fp8_matmul_args* args, ftmoe_stream_t stream);

/* Test hook of ftmoe_fp8_matmul's failure path, like ftmoe_test_withhold_policy.
 * While enabled, a call's first CTA never asks for the tokens of its first
 * block, and the call's waits give up after wait_limit_ns.  The kernel sets the
 * status word's timeout bit and finishes; the tiles of that CTA stay as they
 * were, others come out as usual. */
int ftmoe_test_withhold_matmul(int enable, int64_t wait_limit_ns);

/* h = SiLU(gu[:, :I]) * gu[:, I:] in fp32, for gu [rows, 2I] of `dtype`.
 * scales NULL: out [rows, I] of `dtype`.  Otherwise out is codes [rows, I] and
 * scales [I/128][rows], I a multiple of 128.  `used`: NULL, or the device count
 * of rows to handle; the others stay as they were. */
int ftmoe_swiglu(const void* gu, int dtype, int rows, int I, const int32_t* used, void* out, float* scales,
                 ftmoe_stream_t stream);

/* Its gradient dgu [rows, 2I] from dh [rows, I]; scales NULL: of `dtype`, and
 * may be gu itself.  Otherwise codes and scales [2I/128][rows]. */
int ftmoe_swiglu_backward(const void* dh, const void* gu, int dtype, int rows, int I, const int32_t* used, void* dgu,
                          float* scales, ftmoe_stream_t stream);

/* Synchronise `stream`, read and clear the current device's status word of
 * the training operators and the 8-bit layer since the last call: FTMOE_OK,
 * FTMOE_ERR_DEVICE_CHECK if a kernel met an index out of range, or
 * FTMOE_ERR_TIMEOUT if a bounded wait of the policy loss or of
 * ftmoe_fp8_matmul ran out: that call's outputs are not valid (a loss is NaN as
 * a rule), and the next call starts clean.  One word serves all streams. */
int ftmoe_ops_status(ftmoe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FTMOE_H_ */
