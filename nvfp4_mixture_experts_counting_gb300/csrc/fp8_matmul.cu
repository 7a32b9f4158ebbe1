// Product of E4M3 codes with a scale for each block of 128, grouped by expert:
//   y[r, n] = sum_b sx[b, r] sw[n / 128, b] sum_{k in block b} qx[r, k] qw[n, k]
// with `transpose` by the weights' columns instead (the gradient of the
// input), with `swiglu` h = SwiGLU of y's halves as codes and scales.
//
// Weights are the MMA's 128-row operand and tokens its columns, as many as a
// tile has, rounded up to 16: an expert with a few tokens costs its weights'
// bytes and no empty rows, one with many is cut into equal tiles of at most
// NMAX.  A block's product of 128 x N lands in tensor memory; eight warps read
// it, multiply it by the block's scales and add it up in fp32 registers, while
// the next block's product goes to the other buffer.  (The scales are any
// fp32, so the tensor cores cannot apply them as they do powers of two.)
// tcgen05 sums a block of 128 products in fp32, so an output rounds once per
// block and once at the end.
//
// Warps: 0 copies tiles by TMA, 1 issues the MMAs, 2 multiplies sx by sw into
// shared memory for each block, 4-11 add up.  With SwiGLU a tile is 128 gate
// and the matching 128 up rows, so that a thread has both halves of a value.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp8_common.cuh"
#include "tc_common.cuh"

namespace ftmoe {

namespace {

constexpr int kFewThreads = 256;
constexpr int kManyThreads = 384;
constexpr int kEpiWarp0 = 4;       // the first of the warps that sum
constexpr int kFewWarps = 4, kManyWarps = 8;
// Registers a thread: at launch, of warps 0-3, of the others.
constexpr int kLaunchRegs = 168, kLowRegs = 72, kEpiRegs = 216;
static_assert(3 * kLaunchRegs == kLowRegs + 2 * kEpiRegs, "the warpgroups' shares add up to the launch's registers");
constexpr int kTile = 128 * 128;  // bytes of a weight tile
constexpr int kSmemMax = 227 * 1024;

struct MatmulArgs {
  const float *a_scale, *w_scale;
  const int32_t* offsets;
  int M, E;
  int C, O;        // lengths of an input's and an output's row (with swiglu O is I)
  int NB, KB;      // blocks of the weights' rows and columns
  int JT;          // weight tiles of an expert
  int dtype;
  void* out;
  float* out_scale;
  uint32_t* status;
};

// What a kernel form takes of shared and tensor memory.
template <int NMAX, bool SWIGLU>
struct Form {
  static constexpr int kParts = SWIGLU ? 2 : 1;
  static constexpr int kBox = NMAX < 64 ? 16 : 64;  // tokens of one copy
  static constexpr int kABytes = kParts * kTile, kBBytes = NMAX * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kCols = kParts * NMAX;  // of an accumulator buffer
  static constexpr int kBufs = 512 / kCols < 4 ? 512 / kCols : 4;
  static constexpr int kTmemCols = kBufs * kCols;
  static constexpr int kChunks = NMAX / 32;  // of 32 tokens
  // Staging of a warp's 32 outputs: 16 tokens' in 16 bits, 8 tokens' in fp32 (rows of 36, which keeps the stores'
  // banks apart), or 32 tokens' codes.
  static constexpr int kWarpOut = SWIGLU ? 1024 : 1152;
  static constexpr int kOut = kFewWarps * kWarpOut;
  static constexpr int kTops = SWIGLU ? NMAX * 4 * 4 : 0;  // a token's largest magnitude in each warp
  static constexpr int kScales = kBufs * kCols * 4;
  static constexpr int kFixed = 1024 + kOut + kTops + kScales + 512 + 3 * 4 * (kMaxBins + 1);
  static constexpr int kStages0 = (kSmemMax - kFixed) / kStageBytes;
  static constexpr int kStages = kStages0 < 12 ? kStages0 : 12;
  static constexpr int smem(int E) {
    return 1024 + kStages * kStageBytes + kOut + kTops + kScales + 512 + 3 * 4 * (E + 1);
  }
};

__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_by_columns, bool b_by_columns) {
  return (1u << 4)                             // D: fp32; A and B E4M3 are 0
         | ((a_by_columns ? 1u : 0u) << 15)    // stored by the contracted index
         | ((b_by_columns ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// What the copying and the issuing warps do.  The whole warp runs each with
// the same operands, and one lane, always the same, is elected inside: the
// operands so stay in uniform registers.  Four MMAs take 67 cycles to issue;
// from a branch of one lane, which the compiler cannot know to be uniform,
// they took 208.
#define FTMOE_ELECTED(instruction) "{\n .reg .pred p, q;\n elect.sync _|q, 0xffffffff;\n" instruction "}\n"
__device__ __forceinline__ void elected_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile(FTMOE_ELECTED("@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n") ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void elected_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      FTMOE_ELECTED("@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                    "[%1, {%2, %3}], [%4];\n") ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void elected_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      FTMOE_ELECTED("@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                    "[%1, {%2, %3, %4}], [%5];\n") ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void elected_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(FTMOE_ELECTED("setp.ne.b32 p, %4, 0;\n"
                             " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n") ::"r"(d),
               "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
               : "memory");
}
__device__ __forceinline__ void elected_commit(uint64_t* bar) {
  asm volatile(FTMOE_ELECTED("@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n") ::"r"(
                   smem_u32(bar))
               : "memory");
}

template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A tile of work: tokens [row0, row0 + rows) of expert e times weight tile jt.
struct Unit {
  int e, jt, row0, rows, N;
};

struct Tables {
  const int *start, *count, *first;  // each expert's first row, rows and first unit (first[E]: all)
  int E;
};

// Tables of the experts' rows and units, by the whole CTA.  An expert whose
// rows begin before an earlier one's first row, fall or leave [0, M] has none
// and marks the status word.
template <int NMAX>
__device__ __forceinline__ void make_tables(const MatmulArgs& a, int* start, int* count, int* first) {
  const int E = a.E, lane = threadIdx.x & 31;
  if (a.offsets) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) first[e] = a.offsets[e];
  } else if (threadIdx.x == 0) {
    first[0] = 0;
    first[1] = a.M;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int floor = 0, sum = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const bool on = e < E;
      const int lo = on ? first[e] : 0, hi = on ? first[e + 1] : 0;
      int high = lo;  // the largest start up to this expert
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, high, o);
        if (lane >= o) high = max(high, v);
      }
      high = max(high, floor);
      const bool good = on && lo >= high && hi >= lo && hi <= a.M;
      if (on && !good) set_status(a.status, kStatusRange);
      const int n = good ? hi - lo : 0, units = (n + NMAX - 1) / NMAX * a.JT;
      int upto = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      __syncwarp();  // all have read first[]; the next round reads on from first[e0 + 32]
      if (on) {
        start[e] = lo;
        count[e] = n;
        first[e] = sum + upto - units;
      }
      floor = __shfl_sync(0xffffffffu, high, 31);
      sum += __shfl_sync(0xffffffffu, upto, 31);
      __syncwarp();
    }
    if (lane == 0) first[E] = sum;
  }
  __syncthreads();
}

__device__ __forceinline__ int expert_of(const Tables& t, int u) {
  int lo = 0, hi = t.E;  // the last expert whose first unit is not after u
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;  // experts without units share their successor's first unit: u lies with the last of equals
}

template <int NMAX>
__device__ __forceinline__ Unit unit_of(const Tables& t, int u, int JT) {
  const int lo = expert_of(t, u), n = t.count[lo], tiles = (n + NMAX - 1) / NMAX, r = u - t.first[lo];
  const int jt = r / tiles, nt = r - jt * tiles;
  const int per = ((n + tiles - 1) / tiles + 15) & ~15;
  Unit x;
  x.e = lo;
  x.jt = jt;
  x.row0 = t.start[lo] + nt * per;
  x.rows = min(per, n - nt * per);
  x.N = (x.rows + 15) & ~15;
  return x;
}

// mbar_wait for waits that are mostly over when they begin.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(smem_u32(bar)), "r"(parity), "r"(20000u) : "memory");
    if (done) return true;
    if (globaltimer() - t0 > kWaitLimitNs) {
      set_status(status, kStatusTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  return __all_sync(0xffffffffu, wait(bar, parity, status));
}

// 16 lanes x 32 columns of tensor memory: lane l of the warp gets, of each 8
// columns, the values of row l / 4 in the columns 2 (l % 4) and one more, then
// those of row l / 4 + 8.  Neither this nor the wait orders memory: loads of
// scales may pass them (what they read is ordered by mbarriers).
__device__ __forceinline__ void tc_ld_16x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31]));
}

// Four 8 x 8 matrices of 16-bit values, transposed: a lane holds row l / 4 of
// each, columns 2 (l % 4) and one more; row l % 8 of matrix l / 8 in memory,
// the registers' column, goes to this lane's address.
__device__ __forceinline__ void st_matrix_t(void* p, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(p)), "r"(r0),
               "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

__device__ __forceinline__ uint32_t halves(float lo, float hi, int dtype);
__device__ __forceinline__ uint32_t halves(uint64_t v, int dtype) {
  float lo, hi;
  unpack2(v, lo, hi);
  return halves(lo, hi, dtype);
}
__device__ __forceinline__ uint32_t halves(float lo, float hi, int dtype) {
  if (dtype == FTMOE_FP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int NMAX, bool SWIGLU, bool TRANS>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_fp8_matmul_few(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ CUtensorMap map_x) {
  using F = Form<NMAX, SWIGLU>;
  constexpr int kStages = F::kStages, kBufs = F::kBufs;
  constexpr int kChunks = F::kChunks;
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  unsigned char* staged = sm + kStages * F::kStageBytes;
  uint32_t* tops = reinterpret_cast<uint32_t*>(staged + F::kOut);
  float* s_scale = reinterpret_cast<float*>(staged + F::kOut + F::kTops);
  uint64_t* full = reinterpret_cast<uint64_t*>(staged + F::kOut + F::kTops + F::kScales);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;   // the MMA's commit and the scale warp
  uint64_t* acc_empty = acc_full + kBufs;
  uint64_t* drain = acc_empty + kBufs;
  uint64_t* wg_bar = drain + 1;           // the warps that sum
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(wg_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* t_start = reinterpret_cast<int*>(staged + F::kOut + F::kTops + F::kScales + 512);
  int *t_count = t_start + a.E, *t_first = t_count + a.E;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nkb = (a.C + 127) / 128;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&acc_full[b], 2);
      mbar_init(&acc_empty[b], kFewWarps);
    }
    mbar_init(drain, 1);
    mbar_init(wg_bar, kFewWarps);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_x);
  }
  if (warp == 1) tmem_alloc(tmem_slot, F::kTmemCols);
  pdl_wait();
  make_tables<NMAX>(a, t_start, t_count, t_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Tables tables{t_start, t_count, t_first, a.E};
  const int n_units = t_first[a.E];

  if (warp < kEpiWarp0) {
    if (warp == 0) {
      // ---------------- copies
      int k = 0;
      for (int u = blockIdx.x; u < n_units && !*abort_flag; u += gridDim.x) {
        const Unit x = unit_of<NMAX>(tables, u, a.JT);
        const int boxes = (x.N + F::kBox - 1) / F::kBox;
        for (int kb = 0; kb < nkb; ++kb, ++k) {
          const int s = k % kStages;
          if (k >= kStages && !warp_wait(&empty[s], (k / kStages - 1) & 1, a.status)) {
            *abort_flag = 1;
            break;
          }
          unsigned char* sa = sm + s * F::kStageBytes;
          unsigned char* sb = sa + F::kABytes;
          elected_expect(&full[s], F::kABytes + boxes * F::kBox * 128);
          if (TRANS) {
            elected_load_3d(sa, &map_w, x.jt * 128, kb * 128, x.e, &full[s]);
          } else {
            elected_load_3d(sa, &map_w, kb * 128, x.jt * 128, x.e, &full[s]);
            if (SWIGLU) elected_load_3d(sa + kTile, &map_w, kb * 128, a.O + x.jt * 128, x.e, &full[s]);
          }
          for (int b = 0; b < boxes; ++b)
            elected_load_2d(sb + b * F::kBox * 128, &map_x, kb * 128, x.row0 + b * F::kBox, &full[s]);
        }
      }
      // nothing this warp issued may still be landing when the CTA exits
      for (int q = k > kStages ? k - kStages : 0; q < k; ++q) mbar_wait(&full[q % kStages], (q / kStages) & 1, a.status);
    } else if (warp == 1) {
      // ---------------- products
      int k = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < n_units && !*abort_flag; u += gridDim.x) {
        const Unit x = unit_of<NMAX>(tables, u, a.JT);
        const uint32_t idesc = idesc_e4m3(128, x.N, TRANS, false);
        for (int kb = 0; kb < nkb; ++kb, ++k) {
          const int s = k % kStages, b = k % kBufs;
          if ((k >= kBufs && !warp_wait(&acc_empty[b], (k / kBufs - 1) & 1, a.status)) ||
              !warp_wait(&full[s], (k / kStages) & 1, a.status)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(sm + s * F::kStageBytes);
          const uint64_t adesc = sdesc_k_sw128(sa), bdesc = sdesc_k_sw128(sa + F::kABytes);
          const int steps = (min(128, a.C - kb * 128) + 31) / 32;
          const uint32_t d = tmem + b * F::kCols;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= steps) break;
            // 32 contracted values: 32 bytes on within the swizzled rows, or 32 rows on
            const uint64_t on = TRANS ? i * (32 * 128 >> 4) : i * (32 >> 4);
            elected_mma(d, adesc + on, bdesc + i * (32 >> 4), idesc, i != 0);
            if (SWIGLU) elected_mma(d + NMAX, adesc + on + (kTile >> 4), bdesc + i * (32 >> 4), idesc, i != 0);
          }
          elected_commit(&empty[s]);
          elected_commit(&acc_full[b]);
        }
      }
      elected_commit(drain);
      mbar_wait(drain, 0, a.status);
    } else if (warp == 2) {
      // ---------------- scales: the block's sx sw of each token
      constexpr int kPer = (NMAX + 31) / 32;
      int k = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < n_units && !*abort_flag; u += gridDim.x) {
        const Unit x = unit_of<NMAX>(tables, u, a.JT);
        const float* sx = a.a_scale + x.row0;
        // plain: w_scale[e][jt][kb]; by columns: [e][kb][jt]; the up tile lies O rows on
        const float* sw = a.w_scale + ((int64_t)x.e * a.NB + (TRANS ? 0 : x.jt)) * a.KB + (TRANS ? x.jt : 0);
        const int64_t sw_step = TRANS ? a.KB : 1, up = (int64_t)(a.O / 128) * a.KB;
        float v[kPer], w0 = sw[0], w1 = SWIGLU ? sw[up] : 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = lane + 32 * i < x.rows ? sx[lane + 32 * i] : 0.f;
        for (int kb = 0; kb < nkb; ++kb, ++k) {
          const int b = k % kBufs;
          if (k >= kBufs && !warp_wait(&acc_empty[b], (k / kBufs - 1) & 1, a.status)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          float* to = s_scale + b * F::kCols;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            if (lane + 32 * i >= NMAX) continue;
            to[lane + 32 * i] = v[i] * w0;
            if (SWIGLU) to[NMAX + lane + 32 * i] = v[i] * w1;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_full[b]);
          if (kb + 1 < nkb) {
            const float* next = sx + (int64_t)(kb + 1) * a.M;
            w0 = sw[(kb + 1) * sw_step];
            if (SWIGLU) w1 = sw[up + kb + 1];
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = lane + 32 * i < x.rows ? next[lane + 32 * i] : 0.f;
          }
        }
      }
    }
  } else {
    // ---------------- sums: warp q has TMEM lanes 32q..
    // acc[i][j][m]: chunk i's tokens 8j + 2 (lane % 4) and one more, output 32q + 8m + lane / 4.  A lane so needs
    // the scales of a quarter of the tokens.
    const int q = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    constexpr int kAll = F::kParts * kChunks;
    unsigned char* st = staged + q * F::kWarpOut;
    int k = 0;
    uint32_t wg_phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < n_units && !*abort_flag; u += gridDim.x) {
      const Unit x = unit_of<NMAX>(tables, u, a.JT);
      const int mine = (x.N + 31) / 32;  // chunks there are; the last may be half a one
      uint64_t acc[kAll][4][4];
#pragma unroll
      for (int i = 0; i < kAll; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j / 4][j % 4] = 0ull;
      for (int kb = 0; kb < nkb; ++kb, ++k) {
        const int b = k % kBufs;
        if (!warp_wait(&acc_full[b], (k / kBufs) & 1, a.status)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + lanes + b * F::kCols;
        const float* sc = s_scale + b * F::kCols + 2 * (lane & 3);
#pragma unroll
        for (int i = 0; i < kAll; ++i) {
          if (i % kChunks >= mine) continue;
          // chunk i: part i / kChunks, tokens 32 (i % kChunks)
          const int col = i / kChunks * NMAX + i % kChunks * 32;
          uint32_t r[32];
          tc_ld_16x32(d + col, r);
          tc_ld_16x32(d + col + (16u << 16), r + 16);
          tc_wait32(r);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t s = *reinterpret_cast<const uint64_t*>(sc + col + 8 * j);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint32_t* v = r + 16 * (m / 2) + 4 * j + 2 * (m % 2);
              acc[i][j][m] = fma2(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])), s, acc[i][j][m]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[b]);
      }
      if (!ok) break;
      if constexpr (!SWIGLU) {
        const int o0 = x.jt * 128 + 32 * q, width = min(32, a.O - o0);  // this warp's outputs
        if (a.dtype != FTMOE_FP32) {
          const bool wide = a.O % 8 == 0;
#pragma unroll
          for (int h = 0; h < 2 * kChunks; ++h) {  // by 16 tokens
            const int i = h / 2, j0 = h % 2 * 2, t0 = 32 * i + 16 * (h % 2), rows = min(16, x.rows - t0);
            if (rows <= 0 || width <= 0) continue;
            // [token][32] with the 16-byte pieces of a row turned by the token
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int token = 8 * j + (lane & 7);
              st_matrix_t(st + token * 64 + (((lane / 8) ^ (token / 2 & 3)) << 4), halves(acc[i][j0 + j][0], a.dtype),
                          halves(acc[i][j0 + j][1], a.dtype), halves(acc[i][j0 + j][2], a.dtype),
                          halves(acc[i][j0 + j][3], a.dtype));
            }
            __syncwarp();
            uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)(x.row0 + t0) * a.O + o0;
            if (wide) {
#pragma unroll
              for (int n = lane; n < 64; n += 32) {
                const int token = n >> 2, piece = n & 3;
                if (token < rows && 8 * piece < width)
                  *reinterpret_cast<uint4*>(out + (int64_t)token * a.O + 8 * piece) =
                      *reinterpret_cast<const uint4*>(st + token * 64 + ((piece ^ (token / 2 & 3)) << 4));
              }
            } else if (lane < width) {
              for (int token = 0; token < rows; ++token)
                out[(int64_t)token * a.O + lane] = *reinterpret_cast<const uint16_t*>(
                    st + token * 64 + (((lane >> 3) ^ (token / 2 & 3)) << 4) + 2 * (lane & 7));
            }
          }
        } else {
          const bool wide = a.O % 4 == 0;
          float* to = reinterpret_cast<float*>(st);
#pragma unroll
          for (int h = 0; h < 4 * kChunks; ++h) {  // by 8 tokens
            const int i = h / 4, t0 = 32 * i + 8 * (h % 4), rows = min(8, x.rows - t0);
            if (rows <= 0 || width <= 0) continue;
            __syncwarp();
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              float lo, hi;
              unpack2(acc[i][h % 4][m], lo, hi);
              float* at = to + 2 * (lane & 3) * 36 + 8 * m + lane / 4;
              at[0] = lo;
              at[36] = hi;
            }
            __syncwarp();
            float* out = static_cast<float*>(a.out) + (int64_t)(x.row0 + t0) * a.O + o0;
            if (wide) {
#pragma unroll
              for (int n = lane; n < 64; n += 32) {
                const int token = n >> 3, piece = n & 7;
                if (token < rows && 4 * piece < width)
                  *reinterpret_cast<float4*>(out + (int64_t)token * a.O + 4 * piece) =
                      *reinterpret_cast<const float4*>(to + token * 36 + 4 * piece);
              }
            } else if (lane < width) {
              for (int token = 0; token < rows; ++token) out[(int64_t)token * a.O + lane] = to[token * 36 + lane];
            }
          }
        }
      } else {
        static_assert(!SWIGLU || kChunks == 1, "one chunk of tokens");
        {
          // h in the gate's registers; a token's largest magnitude over the 128 columns from the four warps
          uint32_t* top = tops;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t best0 = 0, best1 = 0;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              float g0, g1, u0, u1;
              unpack2(acc[0][j][m], g0, g1);
              unpack2(acc[kChunks][j][m], u0, u1);
              g0 = g0 * sigmoid(g0) * u0;
              g1 = g1 * sigmoid(g1) * u1;
              best0 = max(best0, magnitude(g0));
              best1 = max(best1, magnitude(g1));
              acc[0][j][m] = pack2(g0, g1);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              best0 = max(best0, __shfl_xor_sync(0xffffffffu, best0, o));
              best1 = max(best1, __shfl_xor_sync(0xffffffffu, best1, o));
            }
            if (lane < 4) {
              top[(8 * j + 2 * lane) * 4 + q] = best0;
              top[(8 * j + 2 * lane + 1) * 4 + q] = best1;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(wg_bar);
          ok = warp_wait(wg_bar, wg_phase, a.status);
          wg_phase ^= 1;
          // lane t works token t's scale out, in each of the four warps
          const uint4 v = reinterpret_cast<const uint4*>(top)[lane];
          const BlockScale s = block_scale(max(max(v.x, v.y), max(v.z, v.w)));
          if (q == 0 && lane < x.rows) a.out_scale[(int64_t)x.jt * a.M + x.row0 + lane] = s.scale;
          const float mul = s.scale == 0.f ? 0.f : s.mul;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int token = 8 * j + 2 * (lane & 3);
            const float m0 = __shfl_sync(0xffffffffu, mul, token), m1 = __shfl_sync(0xffffffffu, mul, token + 1);
            unsigned char* at = st + token * 32 + lane / 4;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              float h0, h1;
              unpack2(acc[0][j][m], h0, h1);
              const uint32_t c = e4m3x4(m0 == 0.f ? 0.f : h0 * m0, m1 == 0.f ? 0.f : h1 * m1, 0.f, 0.f);
              at[8 * m] = (unsigned char)c;
              at[8 * m + 32] = (unsigned char)(c >> 8);
            }
          }
          // the warps meet once more, so that none writes the next tile's `top` before all have read this one's
          __syncwarp();
          if (lane == 0) mbar_arrive(wg_bar);
          ok = warp_wait(wg_bar, wg_phase, a.status) && ok;
          wg_phase ^= 1;
          if (lane < x.rows) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + (int64_t)(x.row0 + lane) * a.O +
                                                  x.jt * 128 + 32 * q);
            const uint4* from = reinterpret_cast<const uint4*>(st + lane * 32);
            out[0] = from[0];
            out[1] = from[1];
          }
        }
      }
      if (!ok) *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, F::kTmemCols);
  }
}

// ---------------------------------------------------------------- many tokens

// Tiles of 128 tokens (the MMA's rows) and 256 weight rows (gate's 128 and the
// matching up's 128 with SwiGLU).  A lane of tensor memory is a token, so a
// thread's scale of a block is one number for all its columns, and no scales
// pass through shared memory.
struct Many {
  static constexpr int kTokens = 128;
  static constexpr int kABytes = kTile, kBBytes = 2 * kTile, kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 4, kBufs = 2, kCols = 256;  // a warp that issues MMAs has a buffer
  static constexpr int kWarpOut = 2048, kOut = kManyWarps * kWarpOut;  // staging: 32 tokens' 64 bytes
  static constexpr int kTops = 128 * 2 * 4;  // a token's largest magnitude in each warpgroup
  static constexpr int kFixed = kOut + kTops;
  static constexpr int smem(int E) { return 1024 + kStages * kStageBytes + kFixed + 512 + 3 * 4 * (E + 1); }
  static_assert(1024 + kStages * kStageBytes + kFixed + 512 + 3 * 4 * (kMaxBins + 1) <= kSmemMax, "");
};

// g / (1 + exp(-g)) by the approximate power of two and reciprocal: within (|g| + 8) 2^-24 of it, while the code that h
// gets is rounded by up to 2^-4.  (The precise forms made a tile's end 9700 cycles long instead of some 3000.)
__device__ __forceinline__ float silu_quick(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return g * r;
}

// 32 lanes x 16 columns of tensor memory, a lane's columns in its registers (see tc_ld_16x32 on memory order).
__device__ __forceinline__ void tc_ld_32x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 32 bytes to a 32-byte-aligned address.
__device__ __forceinline__ void store_32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A warp's sums, lane l those of token l in the columns c0 .. c0 + 127, to the
// rows from `row` on, `rows` of them.  Whole pieces of 32 bytes go straight
// from a lane to its token's row.  Otherwise 64 bytes of every token at a time
// pass through shared memory (`st`), so that a store covers up to eight rows'
// 64 bytes and not 32 rows' few (a product of 666 fp32 columns 60 -> 36 us).
template <bool WIDE>
__device__ __forceinline__ void store_tile(const MatmulArgs& a, unsigned char* st, int64_t row, int rows, int c0,
                                           const float (&acc)[128], int lane) {
  const int bytes = WIDE ? 4 : 2;
  constexpr int kCols = WIDE ? 16 : 32;
  unsigned char* out = static_cast<unsigned char*>(a.out) + (row * a.O + c0) * bytes;
  const int64_t pitch = (int64_t)a.O * bytes;
  if (!WIDE && pitch % 32 == 0 && ((uintptr_t)a.out & 31) == 0 && c0 + 128 <= a.O) {
    if (lane < rows) {
#pragma unroll
      for (int i = 0; i < 128; i += 16) {
        uint32_t p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = halves(acc[i + 2 * j], acc[i + 2 * j + 1], a.dtype);
        store_32(out + lane * pitch + i * bytes, p);
      }
    }
    return;
  }
  const bool aligned = pitch % 16 == 0;
#pragma unroll
  for (int p = 0; p < 128 / kCols; ++p) {
    const int left = (a.O - c0 - p * kCols) * bytes;  // bytes of the row from this piece on
    if (left <= 0) continue;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* v = acc + p * kCols + i * (kCols / 4);
      uint4 w;
      if constexpr (WIDE)
        w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      else
        w = make_uint4(halves(v[0], v[1], a.dtype), halves(v[2], v[3], a.dtype), halves(v[4], v[5], a.dtype),
                       halves(v[6], v[7], a.dtype));
      // the 16-byte pieces of a row turned by the token, against bank conflicts
      *reinterpret_cast<uint4*>(st + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) = w;
    }
    __syncwarp();
    if (aligned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = 8 * i + lane / 4, piece = lane & 3;
        if (token < rows && piece * 16 < left)
          *reinterpret_cast<uint4*>(out + token * pitch + p * 64 + piece * 16) =
              *reinterpret_cast<const uint4*>(st + token * 64 + ((piece ^ (token >> 1 & 3)) << 4));
      }
    } else {
      const int at = lane % kCols * bytes;
      if (at < left) {
        for (int token = lane / kCols; token < rows; token += 32 / kCols) {
          const unsigned char* from = st + token * 64 + (((at >> 4) ^ (token >> 1 & 3)) << 4) + (at & 15);
          unsigned char* to = out + token * pitch + p * 64 + at;
          if constexpr (WIDE)
            *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
          else
            *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(from);
        }
      }
    }
  }
}

template <bool SWIGLU, bool TRANS>
__global__ void __launch_bounds__(kManyThreads, 1)
    k_fp8_matmul_many(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ CUtensorMap map_x) {
  using F = Many;
  constexpr int kStages = F::kStages, kBufs = F::kBufs;
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  unsigned char* staged = sm + kStages * F::kStageBytes;
  uint32_t* tops = reinterpret_cast<uint32_t*>(staged + F::kOut);
  uint64_t* full = reinterpret_cast<uint64_t*>(staged + F::kFixed);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + kBufs;
  uint64_t* drain = acc_empty + kBufs;
  uint64_t* row_bar = drain + 1;  // [4], the warps that hold the same tokens
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(row_bar + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* t_start = reinterpret_cast<int*>(staged + F::kFixed + 512);
  int *t_count = t_start + a.E, *t_first = t_count + a.E;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nkb = (a.C + 127) / 128;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kManyWarps);
    }
    mbar_init(drain, 2);
    for (int w = 0; w < 4; ++w) mbar_init(&row_bar[w], kManyWarps / 4);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_x);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kBufs * F::kCols);
  pdl_wait();
  make_tables<F::kTokens>(a, t_start, t_count, t_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Tables tables{t_start, t_count, t_first, a.E};
  const int n_units = t_first[a.E];
  const auto unit = [&](int u) {
    const int e = expert_of(tables, u), n = t_count[e], tiles = (n + F::kTokens - 1) / F::kTokens, r = u - t_first[e];
    Unit x;
    x.e = e;
    x.jt = r / tiles;
    const int at = (r - x.jt * tiles) * F::kTokens;
    x.row0 = t_start[e] + at;
    x.rows = min(F::kTokens, n - at);
    x.N = F::kCols;
    return x;
  };

  if (warp < kEpiWarp0) {
    regs_down<kLowRegs>();
    if (warp == 0) {
      // ---------------- copies
      int s = 0, k = 0;
      uint32_t phase = 1;
      for (int u = blockIdx.x; u < n_units && !*abort_flag; u += gridDim.x) {
        const Unit x = unit(u);
        for (int kb = 0; kb < nkb; ++kb, ++k) {
          if (!warp_wait(&empty[s], phase, a.status)) {
            *abort_flag = 1;
            break;
          }
          unsigned char* sa = sm + s * F::kStageBytes;
          unsigned char* sb = sa + F::kABytes;
          elected_expect(&full[s], F::kStageBytes);
          elected_load_2d(sa, &map_x, kb * 128, x.row0, &full[s]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int n0 = SWIGLU ? h * a.O + x.jt * 128 : x.jt * 256 + h * 128;
            if (TRANS)
              elected_load_3d(sb + h * kTile, &map_w, n0, kb * 128, x.e, &full[s]);
            else
              elected_load_3d(sb + h * kTile, &map_w, kb * 128, n0, x.e, &full[s]);
          }
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // nothing this warp issued may still be landing when the CTA exits
      for (int q = k > kStages ? k - kStages : 0; q < k; ++q) mbar_wait(&full[q % kStages], (q / kStages) & 1, a.status);
    } else if (warp == 1 || warp == 3) {
      // ---------------- products: warp 1 has the even blocks, warp 3 the odd ones.  Issuing waits while the tensor
      // cores are behind, and what comes between two blocks (the commits, the waits for the next one's buffers) is
      // longer than what they then still have to do; so one warp issues while the other one waits.
      // Few instructions matter here: the summing warps leave few issue slots.
      constexpr uint32_t idesc = idesc_e4m3(F::kTokens, TRANS ? 128 : 256, false, TRANS);
      static_assert(kStages % 2 == 0, "a warp has every other stage");
      // 32 contracted values: 32 bytes on within the swizzled rows, or 32 rows on
      constexpr uint64_t kStepA = 32 >> 4, kStepB = TRANS ? 32 * 128 >> 4 : 32 >> 4;
      const int b = warp >> 1, last_steps = (a.C - (nkb - 1) * 128 + 31) / 32;
      const uint64_t adesc0 = sdesc_k_sw128(smem_u32(sm)), bdesc0 = sdesc_k_sw128(smem_u32(sm) + F::kABytes);
      const uint32_t d = tmem + b * F::kCols;
      int s = b, first = b;  // the stage; this warp's first block of the unit
      uint32_t full_phase = 0, acc_phase = 1;  // a new barrier's phase 1 counts as over
      bool ok = true;
      for (int u = blockIdx.x; ok && u < n_units && !*abort_flag; u += gridDim.x) {
        int kb = first;
        for (; kb < nkb; kb += 2) {
          if (!warp_wait(&acc_empty[b], acc_phase, a.status) || !warp_wait(&full[s], full_phase, a.status)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t adesc = adesc0 + s * (F::kStageBytes >> 4), bdesc = bdesc0 + s * (F::kStageBytes >> 4);
          const int steps = kb == nkb - 1 ? last_steps : 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= steps) break;
            elected_mma(d, adesc + i * kStepA, bdesc + i * kStepB, idesc, i != 0);
            if (TRANS)  // rows of 128 bytes hold 128 columns
              elected_mma(d + 128, adesc + i * kStepA, bdesc + i * kStepB + (kTile >> 4), idesc, i != 0);
          }
          elected_commit(&acc_full[b]);
          elected_commit(&empty[s]);
          acc_phase ^= 1;
          s += 2;
          if (s >= kStages) {
            s -= kStages;
            full_phase ^= 1;
          }
        }
        first = kb - nkb;  // 0 or 1: the blocks of all units are counted on
      }
      elected_commit(drain);
      mbar_wait(drain, 0, a.status);
    }
  } else {
    regs_up<kEpiRegs>();
    // ---------------- sums: warp (wg, q) has tokens 32q.. and the columns [128 wg, 128 wg + 128), with SwiGLU
    // [64 wg, 64 wg + 64) of gate and up.  Packed FMAs: no faster than plain ones here, but half the instructions.
    const int q = warp & 3, wg = (warp - kEpiWarp0) >> 2;
    const uint32_t from = tmem + ((uint32_t)(32 * q) << 16) + (SWIGLU ? 64 : 128) * wg;
    int k = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < n_units && !*abort_flag; u += gridDim.x) {
      const Unit x = unit(u);
      const int token = 32 * q + lane;
      const bool on = token < x.rows;
      const float* sx = a.a_scale + x.row0 + token;
      // weights' scales: [e][block of rows][block of columns]; TRANS contracts the rows
      const int nb = SWIGLU ? x.jt : 2 * x.jt + wg;
      const bool there = nb * 128 < a.O;  // a last tile may have only its first half
      const float* sw = a.w_scale + ((int64_t)x.e * a.NB + (TRANS ? 0 : nb)) * a.KB + (TRANS ? nb : 0);
      const int64_t sw_step = TRANS ? a.KB : 1, up = (int64_t)(a.O / 128) * a.KB;
      uint64_t acc2[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc2[i] = 0ull;
      constexpr int kAhead = 3;
      float v[kAhead], w0[kAhead], w1[kAhead];
      const auto fetch = [&](int kb, int to) {
        if (kb >= nkb) return;
        v[to] = on ? sx[(int64_t)kb * a.M] : 0.f;
        w0[to] = there ? sw[kb * sw_step] : 0.f;
        if (SWIGLU) w1[to] = sw[up + kb];
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i, i);
      for (int kb = 0; kb < nkb; ++kb, ++k) {
        const int b = k & 1;
        const float s0 = v[0] * w0[0], s1 = SWIGLU ? v[0] * w1[0] : s0;
        const uint64_t s2[2] = {pack2(s0, s0), pack2(s1, s1)};
#pragma unroll
        for (int i = 0; i + 1 < kAhead; ++i) {
          v[i] = v[i + 1];
          w0[i] = w0[i + 1];
          if (SWIGLU) w1[i] = w1[i + 1];
        }
        fetch(kb + kAhead, kAhead - 1);
        if (!warp_wait(&acc_full[b], (k >> 1) & 1, a.status)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          uint32_t r[16];
          tc_ld_32x16(from + b * F::kCols + (SWIGLU && h >= 4 ? 128 - 64 : 0) + 16 * h, r);
          if (h == 7) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc2[8 * h + i] =
                fma2(pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), s2[h / 4], acc2[8 * h + i]);
        }
      }
      if (!ok) break;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 64; ++i) unpack2(acc2[i], acc[2 * i], acc[2 * i + 1]);
      if constexpr (!SWIGLU) {
        const int c0 = x.jt * 256 + 128 * wg;
        const int rows = min(32, x.rows - 32 * q);
        unsigned char* st = staged + (warp - kEpiWarp0) * F::kWarpOut;
        if (a.dtype == FTMOE_FP32)
          store_tile<true>(a, st, x.row0 + 32 * q, rows, c0, acc, lane);
        else
          store_tile<false>(a, st, x.row0 + 32 * q, rows, c0, acc, lane);
      } else {
        // a token's 128 values of h lie in the two warps of its rows
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          acc[i] = silu_quick(acc[i]) * acc[64 + i];
          best = max(best, magnitude(acc[i]));
        }
        tops[token * 2 + wg] = best;
        __syncwarp();
        if (lane == 0) mbar_arrive(&row_bar[q]);
        ok = warp_wait(&row_bar[q], phase, a.status);
        phase ^= 1;
        const BlockScale s = block_scale(max(best, tops[token * 2 + (wg ^ 1)]));
        // met once more, so that none writes the next tile's `tops` before all have read this one's
        __syncwarp();
        if (lane == 0) mbar_arrive(&row_bar[q]);
        ok = warp_wait(&row_bar[q], phase, a.status) && ok;
        phase ^= 1;
        if (on) {
          const float mul = s.mul;
          uint8_t* out = static_cast<uint8_t*>(a.out) + (int64_t)(x.row0 + token) * a.O + x.jt * 128 + 64 * wg;
          const bool wide = ((uintptr_t)out & 31) == 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float* f = acc + 32 * h + 4 * i;
              c[i] = s.scale == 0.f ? 0u : e4m3x4(f[0] * mul, f[1] * mul, f[2] * mul, f[3] * mul);
            }
            if (wide) {
              store_32(out + 32 * h, c);
            } else {
              reinterpret_cast<uint4*>(out + 32 * h)[0] = make_uint4(c[0], c[1], c[2], c[3]);
              reinterpret_cast<uint4*>(out + 32 * h)[1] = make_uint4(c[4], c[5], c[6], c[7]);
            }
          }
          if (wg == 0) a.out_scale[(int64_t)x.jt * a.M + x.row0 + token] = s.scale;
        }
      }
      if (!ok) *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kBufs * F::kCols);
  }
}

// ---------------------------------------------------------------- host

cudaError_t encode_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                       const uint32_t* box) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t d[3], st[2];
  cuuint32_t b[3], es[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
  }
  for (int i = 0; i < rank - 1; ++i) st[i] = strides[i];
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), d, st, b, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tensor maps of the weights (boxes of 128 x 128 bytes) and of the rows (`box` of them).
cudaError_t make_maps(const ftmoe_fp8_matmul_args& m, int C, int box, CUtensorMap* map_w, CUtensorMap* map_x) {
  const uint64_t wd[3] = {(uint64_t)m.K, (uint64_t)m.N, (uint64_t)m.E}, ws[2] = {(uint64_t)m.K, (uint64_t)m.N * m.K};
  const uint32_t wb[3] = {128, 128, 1};
  const cudaError_t e = encode_map(map_w, m.w, 3, wd, ws, wb);
  if (e != cudaSuccess) return e;
  const uint64_t xd[2] = {(uint64_t)C, (uint64_t)m.M}, xs[1] = {(uint64_t)C};
  const uint32_t xb[2] = {128, (uint32_t)box};
  return encode_map(map_x, m.a, 2, xd, xs, xb);
}

// `most`: units there may be.
template <typename K>
cudaError_t launch_units(K* k, int threads, const TrainDevice& d, int64_t most, int smem, int smem_max,
                         const MatmulArgs& a, const CUtensorMap& map_w, const CUtensorMap& map_x, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_max);
  if (e != cudaSuccess) return e;
  return launch_after_smem(k, (unsigned)(most < d.num_sms ? most : d.num_sms), threads, smem, s, a, map_w, map_x);
}

template <int NMAX, bool SWIGLU, bool TRANS>
cudaError_t launch_few(const TrainDevice& d, const ftmoe_fp8_matmul_args& m, MatmulArgs a, cudaStream_t s) {
  using F = Form<NMAX, SWIGLU>;
  CUtensorMap map_w, map_x;
  const cudaError_t e = make_maps(m, a.C, F::kBox, &map_w, &map_x);
  if (e != cudaSuccess) return e;
  a.JT = fp8_blocks(a.O);
  return launch_units(k_fp8_matmul_few<NMAX, SWIGLU, TRANS>, kFewThreads, d,
                      (m.M / NMAX + (m.M < m.E ? m.M : m.E)) * a.JT, F::smem(m.E), F::smem(kMaxBins), a, map_w, map_x, s);
}

template <bool SWIGLU, bool TRANS>
cudaError_t launch_many(const TrainDevice& d, const ftmoe_fp8_matmul_args& m, MatmulArgs a, cudaStream_t s) {
  using F = Many;
  CUtensorMap map_w, map_x;
  const cudaError_t e = make_maps(m, a.C, 128, &map_w, &map_x);
  if (e != cudaSuccess) return e;
  a.JT = SWIGLU ? a.O / 128 : (a.O + 255) / 256;
  return launch_units(k_fp8_matmul_many<SWIGLU, TRANS>, kManyThreads, d,
                      (m.M / F::kTokens + (m.M < m.E ? m.M : m.E)) * a.JT, F::smem(m.E), F::smem(kMaxBins), a, map_w, map_x, s);
}

}  // namespace

cudaError_t launch_fp8_matmul(const TrainDevice& d, const ftmoe_fp8_matmul_args& m, cudaStream_t s) {
  MatmulArgs a{};
  a.a_scale = m.a_scale;
  a.w_scale = m.w_scale;
  a.offsets = m.offsets;
  a.M = (int)m.M;
  a.E = m.E;
  a.C = m.transpose ? m.N : m.K;
  a.O = m.transpose ? m.K : m.swiglu ? m.N / 2 : m.N;
  a.NB = fp8_blocks(m.N);
  a.KB = fp8_blocks(m.K);
  a.dtype = m.out_dtype;
  a.out = m.out;
  a.out_scale = m.out_scale;
  a.status = d.status;
  // up to 32 tokens an expert in the mean: narrow tiles, whose stages are nearly all weights
  if (m.M <= (int64_t)32 * m.E) {
    if (m.swiglu) return launch_few<32, true, false>(d, m, a, s);
    return m.transpose ? launch_few<32, false, true>(d, m, a, s) : launch_few<32, false, false>(d, m, a, s);
  }
  if (m.swiglu) return launch_many<true, false>(d, m, a, s);
  return m.transpose ? launch_many<false, true>(d, m, a, s) : launch_many<false, false>(d, m, a, s);
}

}  // namespace ftmoe
