// Clipped policy loss with a KL term, forward and backward from the logits.
//
// With z = logits / temperature, y the row's target and w its weight:
//   logp = z_y - log sum exp z,  r = exp(logp - old),  A the advantage
//   row  = -min(r A, clip(r, 1 - lo, 1 + hi) A) + b (exp(d) - d - 1),  d = ref - logp
//   loss = sum_rows w row
//   dlogits = grad_scale w c / temperature (onehot(y) - softmax z),
//   c = d row / d logp = -A r [r A <= clip(r) A] + b (1 - exp(d))
#include <algorithm>
#include <cfloat>

#include <cooperative_groups.h>

#include "train_common.cuh"

namespace ftmoe {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMinCtas = 6;    // CTAs an SM holds at least, by registers
constexpr int kMaxRanks = 8;   // CTAs of a cluster
constexpr int kUnroll = 4;     // 16-byte pieces a lane sums at a time
constexpr int kChunk = 256;    // 16-byte pieces of one bulk copy
constexpr int kMaxChunks = 16; // of a warp's part
constexpr int kLag = 1;        // chunks between a gradient's departure and the reuse of its buffer
constexpr int kLongThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A running maximum of logits and the sum of 2^(k2 (x - maximum)), k2 =
// log2(e) / temperature.  The maximum is subtracted before the product: a
// fused x k2 - m k2 would leave the rounding of m k2 in every exponent, which
// for logits near the type's lowest value is itself large.
// It starts from -FLT_MAX, so that no difference of two infinities arises
// before a row has a value.
struct MaxSum {
  float m, s;
};
// The joint maximum and sum of a warp's lanes: the maximum first, so that each
// sum is scaled once (ex2.approx is 5e-8 low on average, and lanes joined pair by pair met it at each step).
__device__ __forceinline__ MaxSum warp_join(MaxSum run, float k2) {
  const float m = warp_max_f32(run.m);
  return {m, warp_sum_f32(run.s * exp2_fast((run.m - m) * k2))};
}

__device__ __forceinline__ uint64_t exp2_pair(uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack2(exp2_fast(lo), exp2_fast(hi));
}

// The largest value of a piece, NaN left out (the sum meets it).
template <int N>
__device__ __forceinline__ float pack_max(const Pack<float, N>& x) {
  float m = x.v[0];
#pragma unroll
  for (int e = 1; e < N; ++e) m = fmaxf(m, x.v[e]);
  return m;
}
template <typename H2>
__device__ __forceinline__ H2 max_of_pairs(const H2* p, int n) {
  H2 m = p[0];
#pragma unroll
  for (int e = 1; e < n; ++e) m = __hmax2(m, p[e]);
  return m;
}
template <int N>
__device__ __forceinline__ float pack_max(const Pack<__nv_bfloat16, N>& x) {
  const __nv_bfloat162 m = max_of_pairs(reinterpret_cast<const __nv_bfloat162*>(&x), N / 2);
  return fmaxf(__low2float(m), __high2float(m));
}
template <int N>
__device__ __forceinline__ float pack_max(const Pack<__half, N>& x) {
  const __half2 m = max_of_pairs(reinterpret_cast<const __half2*>(&x), N / 2);
  return fmaxf(__low2float(m), __high2float(m));
}
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> zero_pack() {
  Pack<T, N> r;
#pragma unroll
  for (int e = 0; e < N; ++e) r.set(e, 0.f);
  return r;
}

// One row's 16-byte pieces.  The row starts `skip` values after a 16-byte
// boundary; the first and the last piece may belong to it in part, and are
// then read and written value by value.
template <typename T>
struct Row {
  static constexpr int N = 16 / sizeof(T);
  T* at;  // the boundary
  int skip;
  int end;      // skip + V
  __device__ Row(const T* p, int V) {
    skip = (int)(((uintptr_t)p & 15) / sizeof(T));
    at = const_cast<T*>(p) - skip;
    end = skip + V;
  }
  __device__ int pieces() const { return (int)(((unsigned)end + N - 1) / N); }
  __device__ bool whole(int i) const { return i * N >= skip && end - i * N >= N; }
  __device__ Pack<T, N> load(int i) const {
    if (whole(i)) return load_pack<T, N>(at + (int64_t)i * N);
    Pack<T, N> r;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int e = i * N + c;
      r.set(c, -INFINITY);
      if (e >= skip && e < end) r.v[c] = at[e];
    }
    return r;
  }
  __device__ void store(int i, const Pack<T, N>& r, bool same) const {
    if (same && whole(i)) {
      store_pack<T, N>(at + (int64_t)i * N, r);
      return;
    }
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int e = i * N + c;
      if (e >= skip && e < end) at[e] = r.v[c];
    }
  }
};

// What a row's loss takes besides its logits, and what it gives.
struct RowTerms {
  float row, c;  // the row's loss; its gradient's coefficient, grad_scale w c / temperature
};
__device__ __forceinline__ RowTerms row_terms(const ftmoe_policy_args& a, int64_t n, float w, float logp) {
  const float r = expf(logp - a.old_logp[n]), A = a.advantage[n];
  const float bounded = r < 1.f - a.clip_low ? 1.f - a.clip_low : r > 1.f + a.clip_high ? 1.f + a.clip_high : r;
  const bool clipped = r * A > bounded * A;  // false for NaN, which then reaches the loss and the gradient
  float row = -(clipped ? bounded * A : r * A);
  float c = clipped ? 0.f : -(A * r);
  if (a.ref_logp && a.kl_coef != 0.f) {
    const float d = a.ref_logp[n] - logp, ed = expf(d);
    row += a.kl_coef * (ed - d - 1.f);
    c += a.kl_coef * (1.f - ed);
  }
  return {row, c * (a.grad_scale * w / a.temperature)};
}

__device__ __forceinline__ int64_t target_of(const ftmoe_policy_args& a, int64_t n) {
  return a.id_bytes == 8 ? static_cast<const int64_t*>(a.targets)[n] : static_cast<const int32_t*>(a.targets)[n];
}

// U pieces, 32 apart, join a lane's running maximum and sum.
template <typename T, int U>
__device__ __forceinline__ void add_pieces(const Pack<T, Row<T>::N>* p, float k2, float& m, float& s) {
  constexpr int N = Row<T>::N;
  Pack<T, N> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) x[u] = p[u * 32];
  float top = m;
#pragma unroll
  for (int u = 0; u < U; ++u) top = fmaxf(top, pack_max(x[u]));
  const uint64_t off = pack2(-top, -top), kk = pack2(k2, k2);
  uint64_t sum = pack2(s * exp2_fast((m - top) * k2), 0.f);
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) sum = add2(sum, exp2_pair(mul2(add2(pair_of(x[u], e), off), kk)));
  }
  float a, b;
  unpack2(sum, a, b);
  m = top;
  s = a + b;
}

// U pieces, 32 apart, become -c 2^((x - m) k2 - ls).
template <typename T, int U>
__device__ __forceinline__ void gradient_of_pieces(Pack<T, Row<T>::N>* p, float k2, float m, float ls, float c) {
  constexpr int N = Row<T>::N;
  const uint64_t off = pack2(-m, -m), kk = pack2(k2, k2), down = pack2(-ls, -ls), nc = pack2(-c, -c);
  Pack<T, N> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) x[u] = p[u * 32];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    Pack<T, N> o;
#pragma unroll
    for (int e = 0; e < N / 2; ++e) set_pair(o, e, mul2(exp2_pair(fma2(add2(pair_of(x[u], e), off), kk, down)), nc));
    p[u * 32] = o;
  }
}

// 8 bytes to a peer CTA's shared memory, which complete on its barrier.
__device__ __forceinline__ void send(MaxSum v, MaxSum* slot, uint64_t* bar, int to) {
  uint32_t at, at_bar;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(slot)), "r"(to));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at_bar) : "r"(smem_u32(bar)), "r"(to));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(at), "l"(pack2(v.m, v.s)),
               "r"(at_bar)
               : "memory");
}

// Takes the work of a cluster that has not been launched yet; its first CTA's
// index, or none, arrives in every CTA of this cluster.
__device__ __forceinline__ void ask_for_row(void* response, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], "
      "[%1];" ::"r"(smem_u32(response)),
      "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ bool row_given(const void* response, uint32_t& cta) {
  uint32_t given;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}"
      : "=r"(given), "=r"(cta)
      : "r"(smem_u32(response))
      : "memory");
  return given != 0;
}

// One group of warps takes a row: the warps of a cluster of CTAs, or (SOLO,
// short rows) a single warp.  Each warp copies its part of the row into its
// own shared memory, sums it, and after the group has exchanged its maxima and
// sums, turns it into the gradient in place and sends that off: a row is read
// once and written once, no register holds a load in flight, and the group
// meets once a row.  The copies go in chunks: a chunk is summed while later ones are
// on their way, and as soon as its gradient has left its buffer the next row's
// chunk is asked for.  Clusters take further rows from those not launched yet,
// so rows of weight 0, which cost half or nothing, leave no SM idle.
template <typename T, bool SOLO>
__global__ void __launch_bounds__(kThreads, kMinCtas) k_policy(ftmoe_policy_args a, int part_pieces, uint32_t* status) {
  extern __shared__ __align__(128) unsigned char policy_smem[];
  __shared__ uint64_t bars[kWarps][kMaxChunks];
  __shared__ uint64_t meet[2], ask[2];
  __shared__ __align__(16) uint4 response[2];
  __shared__ MaxSum exchange[2][kMaxRanks * kWarps];
  constexpr int N = Row<T>::N;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = SOLO ? 1 : (int)cluster.num_blocks(), rank = SOLO ? 0 : (int)cluster.block_rank();
  const int log2_ranks = 31 - __clz(ranks);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool first_warp = SOLO || warp == 0, speaks = first_warp && rank == 0 && lane == 0;
  Pack<T, N>* buf = reinterpret_cast<Pack<T, N>*>(policy_smem) + warp * part_pieces;
  T* vals = reinterpret_cast<T*>(buf);
  uint64_t* bar = bars[warp];
  if (lane < kMaxChunks) mbar_init(bar + lane, 1);
  if (!SOLO && threadIdx.x < 2) {
    mbar_init(meet + threadIdx.x, 1);
    mbar_init(ask + threadIdx.x, 1);
  }
  fence_mbar_init();
  __syncwarp();
  const float k2 = kLog2e / a.temperature;
  uint32_t phases = 0;   // of the chunks' barriers
  uint32_t round = 0;    // rows met so far: slot and phase of what the group shares
  bool ok = true;        // no wait has run out

  // This warp's pieces of row n: [lo, hi), the whole ones [wlo, whi).
  struct Part {
    Row<T> z;
    int64_t n;
    int64_t y;
    float w;
    int lo, hi, wlo, whi;
  };
  auto part_of = [&](int64_t n) {
    Part p{Row<T>(static_cast<const T*>(a.logits) + n * a.ld, (int)a.V), n, target_of(a, n),
           a.weight ? a.weight[n] : 1.f / (float)a.N, 0, 0, 0, 0};
    const int pieces = p.z.pieces();
    if (SOLO) {
      p.hi = pieces;
    } else {
      const int per = (pieces + ranks - 1) >> log2_ranks, each = (per + kWarps - 1) / kWarps;
      const int end = min(pieces, (rank + 1) * per);
      p.lo = min(end, rank * per + warp * each);
      p.hi = min(end, p.lo + each);
    }
    p.wlo = max(p.lo, (p.z.skip + N - 1) / N);
    p.whi = max(p.wlo, min(p.hi, p.z.end / N));
    return p;
  };
  auto check = [&](Part& p) {
    if (p.y >= 0 && p.y < a.V) return;
    if (speaks) set_status(status, kStatusRange);
    p.w = 0.f;
  };
  // f(e) for the values e of the pieces that are not whole, among the part's pieces [begin, end).
  auto edges = [&](const Part& p, int begin, int end, auto f) {
    if (lane >= N) return;
    for (int i = p.lo + begin; i < min(p.wlo, p.lo + end); ++i) f(i * N + lane);
    for (int i = max(p.whi, p.lo + begin); i < p.lo + end; ++i) f(i * N + lane);
  };
  // Chunk j of a part, as whole pieces [from, to) (empty: from >= to).
  auto chunk_lo = [&](const Part& p, int j) { return max(p.wlo, p.lo + j * kChunk); };
  auto chunk_hi = [&](const Part& p, int j) { return min(p.whi, p.lo + (j + 1) * kChunk); };
  auto chunks_of = [&](const Part& p) { return (p.hi - p.lo + kChunk - 1) / kChunk; };
  // Asks for a chunk's whole pieces (lane 0).
  auto fetch = [&](const Part& p, int j) {
    const int from = chunk_lo(p, j), to = chunk_hi(p, j);
    if (p.w == 0.f || from >= to) return;
    mbar_arrive_expect_tx(bar + j, (uint32_t)(to - from) * 16);
    bulk_g2s(buf + (from - p.lo), p.z.at + (int64_t)from * N, (uint32_t)(to - from) * 16, bar + j);
  };

  int64_t n = SOLO ? (int64_t)blockIdx.x * kWarps + warp : blockIdx.x >> log2_ranks;
  bool more = n < a.N;
  Part p{Row<T>(nullptr, 0), 0, 0, 0.f, 0, 0, 0, 0};
  if (more) {
    p = part_of(n);
    check(p);
    if (lane == 0)
      for (int j = 0; j < chunks_of(p); ++j) fetch(p, j);
  }
  if (!SOLO) cluster.sync();  // every CTA's barriers are set before a peer uses them
  while (more && ok) {
    const int count = p.hi - p.lo, chunks = chunks_of(p);
    const uint32_t slot = round & 1, turn = round >> 1 & 1;
    if (!SOLO && first_warp && lane == 0) {
      mbar_arrive_expect_tx(ask + slot, 16);
      mbar_arrive_expect_tx(meet + slot, (uint32_t)(ranks * kWarps * sizeof(MaxSum)));
      if (rank == 0) ask_for_row(response + slot, ask + slot);
    }
    float c = 0.f, m = -FLT_MAX, s = 0.f, zy = 0.f;
    if (p.w != 0.f) {
      zy = to_f32(p.z.at[p.z.skip + p.y]);
      if (p.wlo > p.lo || p.whi < p.hi) {
        edges(p, 0, count, [&](int e) {
          vals[e - p.lo * N] = e >= p.z.skip && e < p.z.end ? p.z.at[e] : from_f32<T>(-INFINITY);
        });
        fence_async_smem();
        __syncwarp();
      }
      for (int j = 0; j < chunks; ++j) {
        if (chunk_lo(p, j) < chunk_hi(p, j)) {
          ok = ok && mbar_wait(bar + j, phases >> j & 1, status);
          phases ^= 1u << j;
        }
        const int end = min(count, (j + 1) * kChunk);
        int i = j * kChunk + lane;
        for (; i + 32 * (kUnroll - 1) < end; i += 32 * kUnroll) add_pieces<T, kUnroll>(buf + i, k2, m, s);
        for (; i < end; i += 32) add_pieces<T, 1>(buf + i, k2, m, s);
      }
      // zy is in hand before the group meets: dlogits may be the logits themselves
      if (!ok || isnan(zy)) s = NAN;
    }
    // The next row: its number, and its target and weight on their way while the group meets.
    Part next = p;
    if (SOLO) {
      n += (int64_t)gridDim.x * kWarps;
      more = n < a.N;
    } else {
      uint32_t cta = 0;
      ok = ok && mbar_wait(ask + slot, turn, status);
      more = ok && row_given(response + slot, cta);
      fence_async_smem();  // read before the slot is given again
      n = cta >> log2_ranks;
    }
    if (more) next = part_of(n);

    MaxSum run = warp_join({m, s}, k2);
    if (!SOLO) {
      // Every warp tells every CTA.  Two sets of slots suffice: a warp sends
      // into a set again two rows on, when it has heard in the next row from
      // every warp of the cluster, each after its reads here.
      if (lane < ranks) send(run, &exchange[slot][rank * kWarps + warp], meet + slot, lane);
      ok = mbar_wait(meet + slot, turn, status) && ok;
      run = {-FLT_MAX, 0.f};
      static_assert(kMaxRanks * kWarps <= 32, "a lane a sender");
      if (lane < ranks * kWarps) run = exchange[slot][lane];
      run = warp_join(run, k2);
      if (!ok) run.s = NAN;
    }
    ++round;
    m = run.m;
    const float ls = log2f(run.s);
    if (p.w != 0.f) {
      const float logp = (zy - m) / a.temperature - logf(run.s);
      const RowTerms t = row_terms(a, p.n, p.w, logp);
      c = t.c;
      if (speaks) {
        a.row_loss[p.n] = t.row;
        if (a.logp) a.logp[p.n] = logp;
      }
    } else if (speaks) {
      a.row_loss[p.n] = 0.f;
      if (a.logp) a.logp[p.n] = 0.f;
    }
    if (more) check(next);
    int asked = 0;  // chunks of the next row asked for
    const int next_chunks = more && ok ? chunks_of(next) : 0;
    if (a.dlogits) {
      const Row<T> g(static_cast<T*>(a.dlogits) + p.n * a.ld_d, (int)a.V);
      const bool same = g.skip == p.z.skip;
      T* out = g.at + (g.skip - p.z.skip);  // out[e] belongs to the logit z.at[e]
      const int e0 = max(p.z.skip, p.lo * N), e1 = (int)min((int64_t)p.z.end, (int64_t)p.hi * N);
      if (c == 0.f) {  // nothing of the row's softmax is needed
        __syncwarp();
        if (lane == 0)
          for (; asked < next_chunks; ++asked) fetch(next, asked);
        if (same) {
          for (int i = p.wlo + lane; i < p.whi; i += 32) store_pack<T, N>(out + (int64_t)i * N, zero_pack<T, N>());
          edges(p, 0, count, [&](int e) {
            if (e >= p.z.skip && e < p.z.end) out[e] = from_f32<T>(0.f);
          });
        } else {
          for (int e = e0 + lane; e < e1; e += 32) out[e] = from_f32<T>(0.f);
        }
        asked = next_chunks;
      } else {
        const int target = p.z.skip + (int)p.y - p.lo * N;  // among the part's values
        const float of_target = c * (1.f - exp2_fast((zy - m) * k2 - ls));
        for (int j = 0; j < chunks; ++j) {
          const int begin = j * kChunk, end = min(count, begin + kChunk);
          int i = begin + lane;
          for (; i + 32 * (kUnroll - 1) < end; i += 32 * kUnroll) gradient_of_pieces<T, kUnroll>(buf + i, k2, m, ls, c);
          for (; i < end; i += 32) gradient_of_pieces<T, 1>(buf + i, k2, m, ls, c);
          // the target's own term, by the lane that wrote its piece
          if (target >= begin * N && target < end * N && target / N % 32 == lane) vals[target] = from_f32<T>(of_target);
          fence_async_smem();
          __syncwarp();
          if (!same) continue;
          edges(p, begin, end, [&](int e) {
            if (e >= p.z.skip && e < p.z.end) out[e] = vals[e - p.lo * N];
          });
          if (lane == 0) {
            const int from = chunk_lo(p, j), to = chunk_hi(p, j);
            if (from < to) bulk_s2g(out + (int64_t)from * N, buf + (from - p.lo), (uint32_t)(to - from) * 16);
            bulk_commit();  // one group a chunk, empty or not
            if (j >= kLag) {
              bulk_wait_read<kLag>();  // the gradient of chunk j - kLag has left its buffer
              if (asked < next_chunks) fetch(next, asked++);
            }
          }
        }
        if (!same) {
          for (int e = e0 + lane; e < e1; e += 32) out[e] = vals[e - p.lo * N];
        }
      }
    }
    __syncwarp();
    if (lane == 0) {
      bulk_wait_read<0>();
      for (; asked < next_chunks; ++asked) fetch(next, asked);
    }
    ok = __all_sync(0xffffffffu, ok);
    p = next;
  }
  pdl_launch_dependents();
  if (lane == 0) bulk_wait_read<0>();
  if (!ok) {  // a wait ran out: the copies that may still be on their way
    for (int j = 0; j < chunks_of(p); ++j)
      if (p.w != 0.f && chunk_lo(p, j) < chunk_hi(p, j) && !mbar_wait(bar + j, phases >> j & 1, status)) break;
  }
}

// Rows too long for a cluster's shared memory: the logits are read a second time.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) k_policy_long(ftmoe_policy_args a, uint32_t* status) {
  __shared__ MaxSum warp_part[kLongThreads / 32];
  __shared__ MaxSum exchange[2];
  constexpr int N = Row<T>::N;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float k2 = kLog2e / a.temperature;
  int parity = 0;
  for (int64_t n = blockIdx.x / ranks; n < a.N; n += gridDim.x / ranks) {
    const int64_t y = target_of(a, n);
    float w = a.weight ? a.weight[n] : 1.f / (float)a.N;
    const bool valid = y >= 0 && y < a.V;
    if (!valid && rank == 0 && tid == 0) set_status(status, kStatusRange);
    if (!valid) w = 0.f;
    const Row<T> z(static_cast<const T*>(a.logits) + n * a.ld, (int)a.V);
    const int per = (z.pieces() + ranks - 1) / ranks, lo = min(z.pieces(), rank * per), hi = min(z.pieces(), lo + per);
    float c = 0.f, ls = 0.f, m = 0.f;
    if (w != 0.f) {
      const float zy = to_f32(z.at[z.skip + y]);
      MaxSum run{-FLT_MAX, 0.f};
      for (int i = lo + tid; i < hi; i += kLongThreads) {
        const Pack<T, N> x = z.load(i);
        const float top = fmaxf(run.m, pack_max(x));
        float s = run.s * exp2_fast((run.m - top) * k2);
#pragma unroll
        for (int e = 0; e < N; ++e) s += exp2_fast((x.get(e) - top) * k2);
        run = {top, s};
      }
      run = warp_join(run, k2);
      if (lane == 0) warp_part[warp] = run;
      __syncthreads();
      if (warp == 0) {
        run = warp_join(lane < kLongThreads / 32 ? warp_part[lane] : MaxSum{-FLT_MAX, 0.f}, k2);
        if (lane == 0) exchange[parity] = run;
      }
      cluster.sync();  // two slots suffice, as above
      run = warp_join(lane < ranks ? *cluster.map_shared_rank(&exchange[parity], lane) : MaxSum{-FLT_MAX, 0.f}, k2);
      parity ^= 1;
      m = run.m;
      ls = log2f(run.s);
      const float logp = (zy - m) / a.temperature - logf(run.s);
      const RowTerms t = row_terms(a, n, w, logp);
      c = t.c;
      if (rank == 0 && tid == 0) {
        a.row_loss[n] = t.row;
        if (a.logp) a.logp[n] = logp;
      }
    } else if (rank == 0 && tid == 0) {
      a.row_loss[n] = 0.f;
      if (a.logp) a.logp[n] = 0.f;
    }
    if (!a.dlogits) continue;
    const Row<T> g(static_cast<T*>(a.dlogits) + n * a.ld_d, (int)a.V);
    const bool same = g.skip == z.skip;
    Row<T> out = g;  // at the logits' pieces; of another alignment: written value by value
    out.at += g.skip - z.skip;
    out.skip = z.skip;
    out.end = z.end;
    const int target = z.skip + (int)y;
    for (int i = lo + tid; i < hi; i += kLongThreads) {
      Pack<T, N> o = zero_pack<T, N>();
      if (c != 0.f) {
        const Pack<T, N> x = z.load(i);
#pragma unroll
        for (int e = 0; e < N; ++e)
          o.set(e, c * ((i * N + e == target ? 1.f : 0.f) - exp2_fast(fmaf(x.get(e) - m, k2, -ls))));
      }
      out.store(i, o, same);
    }
  }
  cluster.sync();  // no CTA leaves while a peer may still read its exchange slot
}

// loss = sum_n w_n row_n in a fixed order, by one CTA.
constexpr int kSumThreads = 512;
__global__ void __launch_bounds__(kSumThreads) k_policy_sum(const float* weight, const float* row_loss, int64_t N, float* loss) {
  __shared__ double part[kSumThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  double s = 0.0;
#pragma unroll 4
  for (int64_t n = threadIdx.x; n < N; n += kSumThreads) s += (double)(weight ? weight[n] : 1.f / (float)N) * row_loss[n];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) part[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int w = 0; w < kSumThreads / 32; ++w) s += part[w];
    *loss = (float)s;
  }
}

// A CTA's shared memory for its part of a row: at most, and what lets several CTAs share an SM.
constexpr int kStageMax = 216 * 1024, kStage = 36 * 1024;
constexpr int kSoloBytes = 4096;  // rows up to here are a warp's

}  // namespace

cudaError_t policy_set_limits() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto type) {
    using T = decltype(type);
    const cudaError_t r = cudaFuncSetAttribute(k_policy<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMax);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(k_policy<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMax);
  };
  for (int t : {FTMOE_BF16, FTMOE_FP32, FTMOE_FP16})
    if ((e = with_dtype(t, set)) != cudaSuccess) return e;
  return e;
}

cudaError_t launch_policy_loss(const TrainDevice& d, const ftmoe_policy_args& a, cudaStream_t s) {
  if (a.N > 0) {
    const int bytes = dtype_bytes(a.dtype);
    const int64_t pieces = (a.V * bytes + 15 + 14) / 16;  // of a row at any alignment, at most
    auto part = [&](int ranks) { return ((pieces + ranks - 1) / ranks + kWarps - 1) / kWarps; };  // a warp's pieces
    auto cta_bytes = [&](int ranks) { return part(ranks) * kWarps * 16; };
    const bool solo = pieces * 16 <= kSoloBytes;
    int ranks = 1;
    while (!solo && ranks < kMaxRanks && cta_bytes(ranks) > kStage) ranks *= 2;
    // few rows: spread each over more CTAs while the SMs are not full and a part has work for its warps
    while (!solo && ranks < kMaxRanks && a.N * ranks < 2 * d.num_sms && cta_bytes(ranks) >= 2 * kThreads * 16) ranks *= 2;
    const int64_t smem = solo ? pieces * kWarps * 16 : cta_bytes(ranks);
    cudaLaunchConfig_t c{};
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
    const bool staged = smem <= kStageMax;
    c.blockDim = dim3(staged ? kThreads : kLongThreads);
    c.dynamicSmemBytes = staged ? (size_t)smem : 0;
    const int64_t want = solo ? (a.N + kWarps - 1) / kWarps : a.N;
    const int64_t room = solo ? (int64_t)d.num_sms * 6 : staged ? INT32_MAX / ranks : 1 << 24;  // memory ends before
    c.gridDim = dim3((unsigned)(std::min(want, room) * ranks));
    cudaError_t e = with_dtype(a.dtype, [&](auto type) {
      using T = decltype(type);
      if (!staged) return cudaLaunchKernelEx(&c, k_policy_long<T>, a, d.status);
      const int each = solo ? (int)pieces : (int)part(ranks);
      return solo ? cudaLaunchKernelEx(&c, k_policy<T, true>, a, each, d.status)
                  : cudaLaunchKernelEx(&c, k_policy<T, false>, a, each, d.status);
    });
    if (e != cudaSuccess) return e;
  }
  return launch_after(k_policy_sum, 1, kSumThreads, s, a.weight, a.row_loss, a.N, a.loss);
}

}  // namespace ftmoe
