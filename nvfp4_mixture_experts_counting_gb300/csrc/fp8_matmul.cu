// Product of E4M3 codes with a scale for each block of 128, grouped by expert:
//   y[r, n] = sum_b sx[b, r] sw[n / 128, b] sum_{k in block b} qx[r, k] qw[n, k]
// with `transpose` by the weights' columns instead (the gradient of the
// input), with `swiglu` h = SwiGLU of y's halves as codes and scales.
//
// A unit of work is a tile of an expert's tokens (128, the MMA's rows) times
// 256 of its weight rows (gate's 128 and the matching up's 128 with SwiGLU).
// CTAs walk over the units, an expert's units in order, so that those in
// flight share their weights and tokens in L2.  A block's product of 128 x 256
// lands in one of tensor memory's two buffers; eight warps read it, multiply
// it by the block's scale and add it up in fp32 registers while the next
// block's product goes to the other buffer.  (The scales are any fp32, so the
// tensor cores cannot apply them as they do powers of two.)  A lane of tensor
// memory is a token, so a thread's scale of a block is one number for all its
// columns.  tcgen05 sums a block of 128 products in fp32, so an output rounds
// once per block and once at the end.
//
// What bounds it: with many tokens the summing warps.  A block takes some 1050
// cycles, of which its MMAs are busy 512 (585 from the first issue to the last)
// and a warp's reads and sums 550; the waits for the block and for its scales are
// 120 to 150 each even where nothing is to be waited for, and what other warps
// issue slows those beside them.  16384 tokens of 8 of 256 experts, gate_up [1280,
// 2560] with SwiGLU: 435 us, 1.97 PFLOP/s, in short runs of passes, and 481 in long
// ones, which meet the power limit; its input's gradient 516 and 548; down 328; one
// matrix of 4096 x 4096 with 4096 rows 70 us, 1.96 PFLOP/s.  With few tokens the
// weights' bytes: 256 tokens of the same layer 137 us, 6.0 TB/s; 16 tokens 50 us,
// 5.0 TB/s (units of uneven experts over 152 SMs).
//
// So the copies are spread: one of 128 tokens where experts have that many (32
// otherwise: the smaller copies read less of the next expert's rows; 16384 tokens
// with SwiGLU 436 instead of 465 us), weights by one warp and tokens by another,
// on different schedulers, and the scales through shared memory by the second
// (loaded by the summing warps three blocks ahead: the input's gradient 539, down
// 344, gate_up without SwiGLU 473 instead of 446 us).
//
// Measured and not kept, each against the kernel of its time in short runs, in
// which some 9 us are the events': tokens as the MMA's columns (scales then differ by
// column: 955 us); CTA pairs on one 256-token tile (the MMAs run at 530 cycles,
// but the hand-offs cross CTAs and a quarter of the rows are empty: 512 us);
// 16 summing warps of 64 columns (543 us when one warp made all copies); reads of
// 32 columns of tensor memory (537 us).
// For few tokens: narrow tiles of the tokens as columns (64 tokens through down
// 80 us, 68 without), pairs of CTAs that share a unit's blocks (16 tokens through
// gate_up 76 us, 58 without; the exchange of sums costs more than idle SMs).
//
// Warps: 0 copies the weights' tiles by TMA, 2 the tokens' and the scales, 1 and 3
// issue the MMAs, 4-11 add up.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp8_common.cuh"
#include "tc_common.cuh"

namespace ftmoe {

namespace {

constexpr int kThreads = 384;
constexpr int kSumWarp0 = 4;  // the first of the eight that sum
// Registers a thread: at launch, of warps 0-3, of the summing ones.
constexpr int kLaunchRegs = 168, kLowRegs = 72, kSumRegs = 216;
static_assert(3 * kLaunchRegs == kLowRegs + 2 * kSumRegs, "the warpgroups' shares add up to the launch's registers");
constexpr int kTile = 128 * 128;  // bytes of 128 rows of a block
constexpr int kSmemMax = 227 * 1024;
constexpr int kBufs = 2, kCols = 256;  // accumulators: a warp that issues MMAs has one

struct MatmulArgs {
  const float *a_scale, *w_scale;
  const int32_t* offsets;
  int M, E;
  int C, O;    // lengths of an input's and an output's row (with swiglu O is I)
  int NB, KB;  // blocks of the weights' rows and columns
  int JT;      // weight tiles of an expert
  int dtype;
  int box;      // tokens of one copy: 32, or 128
  int map_out;  // rows are whole 16 bytes: tiles may go out by TMA
  void* out;
  float* out_scale;
  uint32_t* status;
  uint32_t wait_ns;  // limit of a wait
  int withhold;      // a test's: the first CTA never asks for its first block's tokens and scales
};

constexpr int kTokens = 128;
constexpr int kStageBytes = 3 * kTile, kStages = 4;  // a block's tokens and 256 weight rows
constexpr int kBox = 32;                             // tokens of one copy
constexpr int kStaged = 2048, kOut = 8 * kStaged;    // of a summing warp: 64 bytes of 32 tokens
constexpr int kTops = kTokens * 2 * 4;               // a token's largest magnitude in each warpgroup
// Scales of a block on their way through shared memory: its tokens' and two of the weights'.  A slot is written
// once the MMAs of the block four before are done, hence the sums of the block six before.
constexpr int kScaleSlots = 8, kScaleBytes = (kTokens + 4) * 4;
static_assert(kScaleSlots >= kStages + kBufs, "");
constexpr int kFixed = kOut + kTops + kScaleSlots * kScaleBytes;
constexpr int smem_bytes(int E) { return 1024 + kStages * kStageBytes + kFixed + 512 + 2 * 4 * (E + 1); }
static_assert(smem_bytes(kMaxBins) <= kSmemMax, "");

// Tokens K-major; the weights too, or with `columns` stored by the contracted index.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool columns) {
  return (1u << 4)  // D: fp32; A and B E4M3 are 0
         | ((columns ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
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

// 4 bytes to shared memory behind the warp's back; the barrier gets an arrival from each lane when its copies are there.
__device__ __forceinline__ void copy_4(void* to, const float* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void arrive_copied(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A unit: tokens [row0, row0 + rows) of expert e times weight tile jt.
struct Unit {
  int e, jt, row0, rows;
};

struct Tables {
  const int *start, *first;  // [E + 1]: each expert's first row (the offsets) and first unit
  int E;
};

// Token tiles of n rows, n up to the largest int.
__device__ __forceinline__ int tiles_of(int n) { return n > 0 ? (n - 1) / kTokens + 1 : 0; }

// Tables of the experts' rows and units, by the whole CTA.  An expert whose
// rows begin before an earlier one's first row, fall or leave [0, M] has no
// units and marks the status word.
__device__ __forceinline__ void make_tables(const MatmulArgs& a, int* start, int* first) {
  const int E = a.E, lane = threadIdx.x & 31;
  if (a.offsets) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) start[e] = a.offsets[e];
  } else if (threadIdx.x == 0) {
    start[0] = 0;
    start[1] = a.M;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int floor = 0, sum = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const bool on = e < E;
      const int lo = on ? start[e] : 0, hi = on ? start[e + 1] : 0;
      int high = lo;  // the largest start up to this expert
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, high, o);
        if (lane >= o) high = max(high, v);
      }
      high = max(high, floor);
      const bool good = on && lo >= high && hi >= lo && hi <= a.M;
      if (on && !good) set_status(a.status, kStatusRange);
      const int units = good ? tiles_of(hi - lo) * a.JT : 0;
      int upto = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      if (on) first[e] = sum + upto - units;
      floor = __shfl_sync(0xffffffffu, high, 31);
      sum += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) first[E] = sum;
  }
  __syncthreads();
}

// Unit u, whose expert is not before e.  An expert's units go by weight tile,
// and token tile by token tile within one: CTAs side by side read the same 32
// KB of weights and their own 16 KB of tokens of each block.  (The other way
// round a product of 4096^3 took 84 us instead of 76.)
__device__ __forceinline__ Unit unit_of(const Tables& t, int u, int e) {
  // the last expert whose first unit is not after u (those without units share their successor's), in growing steps
  // from e, then by halves
  int step = 1;
  while (e + step < t.E && t.first[e + step] <= u) {
    e += step;
    step *= 2;
  }
  for (int hi = min(e + step, t.E); hi - e > 1;) {
    const int mid = (e + hi) >> 1;
    if (t.first[mid] <= u) e = mid; else hi = mid;
  }
  const int n = t.start[e + 1] - t.start[e], tiles = tiles_of(n), r = u - t.first[e];
  const int jt = r / tiles, at = (r - jt * tiles) * kTokens;
  return {e, jt, t.start[e] + at, min(kTokens, n - at)};
}

// mbar_wait for waits that are mostly over when they begin.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const MatmulArgs& a) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(smem_u32(bar)), "r"(parity), "r"(20000u) : "memory");
    if (done) return true;
    if (globaltimer() - t0 > a.wait_ns) {
      set_status(a.status, kStatusTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const MatmulArgs& a) {
  return __all_sync(0xffffffffu, wait(bar, parity, a));
}
// Has a wait of the CTA run out?  The lanes agree: one that left its loop alone would leave the others waiting for it.
__device__ __forceinline__ bool given_up(const volatile int* flag) { return __any_sync(0xffffffffu, *flag); }

__device__ __forceinline__ uint32_t halves(float lo, float hi, int dtype) {
  if (dtype == FTMOE_FP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// g / (1 + exp(-g)) by the approximate power of two and reciprocal, relative to it within (1.25 |g| + 8) 2^-24: the
// exponent's rounding (|g|) and that of its constant (0.23 |g|), the power (4), the sum (1), the reciprocal (2) and the
// product (1).  Below -87.3 the reciprocal is flushed to zero.  The code that h gets is rounded by up to 2^-4.  (The
// precise forms made a tile's end 9700 cycles long instead of some 3000.)
__device__ __forceinline__ float silu_quick(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return g * r;
}

// 32 lanes x 16 columns of tensor memory, a lane's columns in its registers, which are there after tc_wait (see
// tc_ld_16x32 on memory order).
__device__ __forceinline__ void tc_ld_32x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The registers pass through it, so that no use of them moves before it.
__device__ __forceinline__ void tc_wait(uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
        "+r"(r[14]), "+r"(r[15]));
}

// 32 bytes to a 32-byte-aligned address.
__device__ __forceinline__ void store_32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A warp's sums, lane l those of token l in the columns c0 .. c0 + 127, to the
// rows from `row` on, `rows` of them, through shared memory (`st`).  A whole 32
// of aligned rows (`map`) go out by TMA behind the warp's back: stores of its
// own pass a 32-byte sector a cycle, 2200 cycles for a tile's 64 KB, in which
// the tensor cores come to a stop (16384 tokens through down 361 us, and 342 with
// the copies).  Others go as stores that cover up to eight rows' 64 bytes each,
// and not 32 rows' few (a product of 666 fp32 columns 60 -> 34 us).
template <bool WIDE>
__device__ __forceinline__ void store_tile(const MatmulArgs& a, unsigned char* st, int64_t row, int rows, int c0,
                                           const float (&acc)[128], int lane, const CUtensorMap* map) {
  const int bytes = WIDE ? 4 : 2;
  constexpr int kCols = WIDE ? 16 : 32;
  unsigned char* out = static_cast<unsigned char*>(a.out) + (row * a.O + c0) * bytes;
  const int64_t pitch = (int64_t)a.O * bytes;
  if (map && rows == 32) {
    // 32 bytes of every token at a time, two pieces in turn, copied out behind the warp's back
    constexpr int kPiece = WIDE ? 8 : 16;
#pragma unroll
    for (int p = 0; p < 128 / kPiece; ++p) {
      if (c0 + p * kPiece >= a.O) continue;
      unsigned char* to = st + (p & 1) * 1024;
      // the tile before may have ended with either piece
      if (lane == 0) p == 0 ? bulk_wait_read<0>() : bulk_wait_read<1>();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* v = acc + p * kPiece + i * (kPiece / 2);
        uint4 w;
        if constexpr (WIDE)
          w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else
          w = make_uint4(halves(v[0], v[1], a.dtype), halves(v[2], v[3], a.dtype), halves(v[4], v[5], a.dtype),
                         halves(v[6], v[7], a.dtype));
        *reinterpret_cast<uint4*>(to + lane * 32 + ((i ^ (lane >> 2 & 1)) << 4)) = w;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(c0 + p * kPiece), "r"((int)row), "r"(smem_u32(to))
                     : "memory");
        bulk_commit();
      }
    }
    return;
  }
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
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
__global__ void __launch_bounds__(kThreads, 1)
    k_fp8_matmul(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_out) {
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  unsigned char* staged = sm + kStages * kStageBytes;
  uint32_t* tops = reinterpret_cast<uint32_t*>(staged + kOut);
  float* scales = reinterpret_cast<float*>(staged + kOut + kTops);
  uint64_t* full = reinterpret_cast<uint64_t*>(staged + kFixed);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + kBufs;
  uint64_t* drain = acc_empty + kBufs;
  uint64_t* row_bar = drain + 1;  // [4], the warps that hold the same tokens
  uint64_t* scaled = row_bar + 4;  // [kScaleSlots]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scaled + kScaleSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int *t_start = reinterpret_cast<int*>(staged + kFixed + 512), *t_first = t_start + a.E + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nkb = (a.C + 127) / 128;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);
    }
    mbar_init(drain, 2);
    for (int w = 0; w < 4; ++w) mbar_init(&row_bar[w], 2);
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(&scaled[i], 32);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_x);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kBufs * kCols);
  pdl_wait();
  make_tables(a, t_start, t_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Tables tables{t_start, t_first, a.E};
  const int n_units = t_first[a.E];

  if (warp < kSumWarp0) {
    regs_down<kLowRegs>();
    if (warp == 0 || warp == 2) {
      // ---------------- copies: warp 0 has the weights, warp 2 the tokens and the scales
      const bool withhold = a.withhold && blockIdx.x == 0;
      int s = 0, k = 0, e = 0;
      uint32_t phase = 1;  // a new barrier's phase 1 counts as over
      for (int u = blockIdx.x; u < n_units && !given_up(abort_flag); u += gridDim.x) {
        const Unit x = unit_of(tables, u, e);
        e = x.e;
        const int boxes = (x.rows + a.box - 1) / a.box;  // the rows behind them in shared memory are nobody's
        // this lane's tokens' scales, and of lanes 0 and 1 the weights' ([e][block of rows][block of columns]; TRANS
        // contracts the rows)
        const int nb = SWIGLU ? x.jt + lane * (a.O / 128) : 2 * x.jt + lane;
        const bool mine = lane < 2 && (SWIGLU || nb * 128 < a.O);  // a last tile may have only its first half
        const int w_step = TRANS ? a.KB : 1;
        const float* from_x = a.a_scale + x.row0 + lane;
        const float* from_w = a.w_scale + ((int64_t)x.e * a.NB + (TRANS ? 0 : nb)) * a.KB + (TRANS ? nb : 0);
        for (int kb = 0; kb < nkb; ++kb, ++k) {
          if (!warp_wait(&empty[s], phase, a)) {
            *abort_flag = 1;
            break;
          }
          unsigned char* sx = sm + s * kStageBytes;
          unsigned char* sw = sx + kTile;
          if (warp == 0) {
            elected_expect(&full[s], 2 * kTile);
            if constexpr (SWIGLU) {
              elected_load_3d(sw, &map_w, kb * 128, x.jt * 128, x.e, &full[s]);
              elected_load_3d(sw + kTile, &map_w, kb * 128, a.O + x.jt * 128, x.e, &full[s]);
            } else if constexpr (TRANS) {
              elected_load_3d(sw, &map_w, x.jt * 256, kb * 128, x.e, &full[s]);
              elected_load_3d(sw + kTile, &map_w, x.jt * 256 + 128, kb * 128, x.e, &full[s]);
            } else {
              elected_load_3d(sw, &map_w, kb * 128, x.jt * 256, x.e, &full[s]);
            }
          } else if (k > 0 || !withhold) {
            elected_expect(&full[s], boxes * a.box * 128);
            for (int i = 0; i < boxes; ++i)
              elected_load_2d(sx + i * a.box * 128, &map_x, kb * 128, x.row0 + i * a.box, &full[s]);
            float* sc = scales + k % kScaleSlots * (kScaleBytes / 4);
#pragma unroll
            for (int i = 0; i < kTokens; i += 32)
              if (lane + i < x.rows) copy_4(sc + lane + i, from_x + i);
            if (mine) copy_4(sc + kTokens + lane, from_w);
            arrive_copied(&scaled[k % kScaleSlots]);
          }
          from_x += a.M;
          from_w += w_step;
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // nothing this warp issued may still be landing when the CTA exits
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (int q = k > kStages ? k - kStages : 0; q < k; ++q) mbar_wait(&full[q % kStages], (q / kStages) & 1, a.status, a.wait_ns);
    } else if (warp == 1 || warp == 3) {
      // ---------------- products: warp 1 has the even blocks, warp 3 the odd ones.  Issuing waits while the tensor
      // cores are behind, and what comes between two blocks (the commits, the waits for the next one's buffers) is
      // longer than what they then still have to do; so one warp issues while the other one waits.  Few instructions
      // matter here: the summing warps leave few issue slots.
      constexpr uint32_t idesc = idesc_e4m3(128, TRANS ? 128 : 256, TRANS);
      static_assert(kStages % 2 == 0, "a warp has every other stage");
      // 32 contracted values: 32 bytes on within the swizzled rows, or 32 rows on
      constexpr uint64_t kStepX = 32 >> 4, kStepW = TRANS ? 32 * 128 >> 4 : 32 >> 4;
      const int b = warp >> 1, last_steps = (a.C - (nkb - 1) * 128 + 31) / 32;
      const uint64_t xdesc0 = sdesc_k_sw128(smem_u32(sm)), wdesc0 = sdesc_k_sw128(smem_u32(sm) + kTile);
      const uint32_t d = tmem + b * kCols;
      int s = b, first = b;  // the stage; this warp's first block of the unit
      uint32_t full_phase = 0, acc_phase = 1;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < n_units && !given_up(abort_flag); u += gridDim.x) {
        int kb = first;
        for (; kb < nkb; kb += 2) {
          if (!warp_wait(&acc_empty[b], acc_phase, a) || !warp_wait(&full[s], full_phase, a)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t xdesc = xdesc0 + s * (kStageBytes >> 4), wdesc = wdesc0 + s * (kStageBytes >> 4);
          const int steps = kb == nkb - 1 ? last_steps : 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= steps) break;
            elected_mma(d, xdesc + i * kStepX, wdesc + i * kStepW, idesc, i != 0);
            if (TRANS)  // rows of 128 bytes hold 128 columns
              elected_mma(d + 128, xdesc + i * kStepX, wdesc + i * kStepW + (kTile >> 4), idesc, i != 0);
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
      mbar_wait(drain, 0, a.status, a.wait_ns);
    }
  } else {
    regs_up<kSumRegs>();
    // ---------------- sums: warp (wg, q) has tokens 32q.. and the columns [128 wg, 128 wg + 128), with SwiGLU
    // [64 wg, 64 wg + 64) of gate and up.  Packed FMAs: no faster than plain ones here, but half the instructions.
    const int q = warp & 3, wg = (warp - kSumWarp0) >> 2, token = 32 * q + lane;
    const uint32_t from = tmem + ((uint32_t)(32 * q) << 16) + (SWIGLU ? 64 : 128) * wg;
    int k = 0, e = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < n_units && !given_up(abort_flag); u += gridDim.x) {
      const Unit x = unit_of(tables, u, e);
      e = x.e;
      const bool on = token < x.rows;
      uint64_t acc2[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc2[i] = 0ull;
      for (int kb = 0; kb < nkb; ++kb, ++k) {
        const int b = k & 1;
        if (!warp_wait(&scaled[k % kScaleSlots], k / kScaleSlots & 1, a)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        const float* sc = scales + k % kScaleSlots * (kScaleBytes / 4);
        const float v = sc[token], s0 = v * sc[kTokens + (SWIGLU ? 0 : wg)], s1 = SWIGLU ? v * sc[kTokens + 1] : s0;
        const uint64_t s2[2] = {pack2(s0, s0), pack2(s1, s1)};
        if (!warp_wait(&acc_full[b], (k >> 1) & 1, a)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        // 16 columns are on their way while 16 are added (the input's gradient 547 -> 543 us, down 346 -> 342)
        uint32_t r[2][16];
        const auto column = [&](int h) { return from + b * kCols + (SWIGLU && h >= 4 ? 128 - 64 : 0) + 16 * h; };
        tc_ld_32x16(column(0), r[0]);
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          tc_wait(r[h & 1]);
          if (h < 7) tc_ld_32x16(column(h + 1), r[h + 1 & 1]);
          if (h == 7) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc2[8 * h + i] = fma2(pack2(__uint_as_float(r[h & 1][2 * i]), __uint_as_float(r[h & 1][2 * i + 1])), s2[h / 4],
                                   acc2[8 * h + i]);
        }
      }
      if (!ok) break;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 64; ++i) unpack2(acc2[i], acc[2 * i], acc[2 * i + 1]);
      if constexpr (!SWIGLU) {
        const int c0 = x.jt * 256 + 128 * wg, rows = min(32, x.rows - 32 * q);
        unsigned char* st = staged + (warp - kSumWarp0) * kStaged;
        if (a.dtype == FTMOE_FP32)
          store_tile<true>(a, st, (int64_t)x.row0 + 32 * q, rows, c0, acc, lane, a.map_out ? &map_out : nullptr);
        else
          store_tile<false>(a, st, (int64_t)x.row0 + 32 * q, rows, c0, acc, lane, a.map_out ? &map_out : nullptr);
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
        ok = warp_wait(&row_bar[q], phase, a);
        phase ^= 1;
        const BlockScale s = block_scale(max(best, tops[token * 2 + (wg ^ 1)]));
        // met once more, so that none writes the next tile's `tops` before all have read this one's
        __syncwarp();
        if (lane == 0) mbar_arrive(&row_bar[q]);
        ok = warp_wait(&row_bar[q], phase, a) && ok;
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
    if (!SWIGLU && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kBufs * kCols);
  }
}

// ---------------------------------------------------------------- host

cudaError_t encode_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                       const uint32_t* box, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8,
                       CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
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
  const CUresult r = fn(m, type, rank, const_cast<void*>(base), d, st, b, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t fp8_matmul_set_limits() {
  const cudaFuncAttribute what = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(k_fp8_matmul<false, false>, what, kSmemMax);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_fp8_matmul<false, true>, what, kSmemMax);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_fp8_matmul<true, false>, what, kSmemMax);
  return e;
}

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
  a.JT = m.swiglu ? a.O / 128 : (a.O + 255) / 256;
  a.dtype = m.out_dtype;
  a.out = m.out;
  a.out_scale = m.out_scale;
  a.status = d.status;
  a.wait_ns = d.test_matmul_ns ? d.test_matmul_ns : (uint32_t)kWaitLimitNs;
  a.withhold = d.test_matmul_ns != 0;
  CUtensorMap map_w, map_x;
  const uint64_t wd[3] = {(uint64_t)m.K, (uint64_t)m.N, (uint64_t)m.E}, ws[2] = {(uint64_t)m.K, (uint64_t)m.N * m.K};
  const uint32_t wb[3] = {128, m.swiglu || m.transpose ? 128u : 256u, 1};
  cudaError_t e = encode_map(&map_w, m.w, 3, wd, ws, wb);
  if (e != cudaSuccess) return e;
  const uint64_t xd[2] = {(uint64_t)a.C, (uint64_t)m.M}, xs[1] = {(uint64_t)a.C};
  a.box = m.M / m.E >= kTokens ? kTokens : kBox;
  const uint32_t xb[2] = {128, (uint32_t)a.box};
  if ((e = encode_map(&map_x, m.a, 2, xd, xs, xb)) != cudaSuccess) return e;
  CUtensorMap map_out = map_x;
  if (!m.swiglu) {
    const int size = m.out_dtype == FTMOE_FP32 ? 4 : 2;
    a.map_out = (int64_t)a.O * size % 16 == 0;
    if (a.map_out) {
      const uint64_t od[2] = {(uint64_t)a.O, (uint64_t)m.M}, os[1] = {(uint64_t)a.O * size};
      const uint32_t ob[2] = {(uint32_t)(32 / size), 32};
      e = encode_map(&map_out, m.out, 2, od, os, ob,
                     size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                     CU_TENSOR_MAP_SWIZZLE_32B);
      if (e != cudaSuccess) return e;
    }
  }
  const int64_t units = (m.M / kTokens + (m.M < m.E ? m.M : m.E)) * a.JT;  // at most
  return launch_after_smem(m.swiglu ? k_fp8_matmul<true, false> : m.transpose ? k_fp8_matmul<false, true>
                                                                              : k_fp8_matmul<false, false>,
                           (unsigned)(units < d.num_sms ? units : d.num_sms), kThreads, smem_bytes(m.E), s, a, map_w,
                           map_x, map_out);
}

}  // namespace ftmoe
