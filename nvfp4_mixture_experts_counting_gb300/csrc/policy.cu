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

constexpr int kMinWarps = 24;    // an SM holds at least, by registers
constexpr int kWarps = 4;        // of a CTA (k_policy: at most)
constexpr int kMaxRanks = 8;     // CTAs of a cluster
constexpr int kUnroll = 4;       // 16-byte pieces a lane sums at a time
constexpr int kChunk = 256;      // 16-byte pieces of one bulk copy
constexpr int kMaxChunks = 14;   // of a warp's part
constexpr int kShortChunks = 2;  // of a short row
constexpr int kLag = 1;          // chunks between a gradient's departure and the reuse of its buffer
constexpr int kLongThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
// sum is scaled once, and by expf: ex2.approx is 5e-8 low on average, which a
// row's every term would meet at each join.
__device__ __forceinline__ MaxSum warp_join(MaxSum run, float k2) {
  const float m = warp_max_f32(run.m);
  return {m, warp_sum_f32(run.s * expf((run.m - m) * (k2 * kLn2)))};
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

// What a row's loss takes besides its logits.
struct RowInputs {
  int64_t n, y;
  float w, old, ref, adv;
};
__device__ __forceinline__ RowInputs row_inputs(const ftmoe_policy_args& a, int64_t n) {
  return {n, a.id_bytes == 8 ? static_cast<const int64_t*>(a.targets)[n] : static_cast<const int32_t*>(a.targets)[n],
          a.weight ? a.weight[n] : 1.f / (float)a.N, a.old_logp[n], a.ref_logp ? a.ref_logp[n] : 0.f, a.advantage[n]};
}
// A row whose target is out of range is marked (by one thread) and counts nothing.
__device__ __forceinline__ void check_target(const ftmoe_policy_args& a, RowInputs& r, bool speaks, uint32_t* status) {
  if (r.y >= 0 && r.y < a.V) return;
  if (speaks) set_status(status, kStatusRange);
  r.w = 0.f;
}

// A log probability as the sum of two fp32 values: rows' losses are of either
// sign and largely cancel in their sum, so the rounding of a value near 10
// (5e-7) is kept out of the ratio and the KL term.
struct LogProb {
  float hi, lo;
  __device__ __forceinline__ float value() const { return hi + lo; }
  // this - v, for a v near it
  __device__ __forceinline__ float minus(float v) const { return (hi - v) + lo; }
};
// a + b as its rounded value and the rounding (0 where that says nothing).
__device__ __forceinline__ LogProb exact_sum(float a, float b) {
  const float t = __fadd_rn(a, b), u = __fsub_rn(t, a);
  const float e = __fadd_rn(__fsub_rn(a, __fsub_rn(t, u)), __fsub_rn(b, u));
  return {t, isfinite(t) ? e : 0.f};
}
// (zy - m) / T - ln s.  One Newton step each, q + (d - q T) / T for the quotient
// and ln s = y + (s e^-y - 1), brings their errors to those of a product and of expf.
__device__ __forceinline__ LogProb log_prob(float zy, float m, float s, float temperature, float inv_t) {
  const LogProb d = exact_sum(zy, -m);
  const float q = d.hi * inv_t;
  const float rest = isfinite(q) ? (fmaf(-q, temperature, d.hi) + d.lo) * inv_t : 0.f;
  const float y = logf(s), dy = fmaf(s, expf(-y), -1.f);
  LogProb r = exact_sum(q, -y);
  r.lo += rest - dy;
  return r;
}

// exp(d) - 1 - d, and e = exp(d) - 1.  Near the reference both differences
// cancel (of exp(d) - d - 1 nothing is left at |d| = 3e-4), so up to |d| = 1 they
// come from the series d^2 (1/2! + d/3! + ... + d^9/11!), whose rest is 2^-27 of
// it; it is never negative.
__device__ __forceinline__ float kl_term(float d, float& e) {
  if (!(fabsf(d) < 1.f)) {
    e = expf(d) - 1.f;
    return e - d;
  }
  float s = 1.f / 39916800.f;
  s = fmaf(s, d, 1.f / 3628800.f);
  s = fmaf(s, d, 1.f / 362880.f);
  s = fmaf(s, d, 1.f / 40320.f);
  s = fmaf(s, d, 1.f / 5040.f);
  s = fmaf(s, d, 1.f / 720.f);
  s = fmaf(s, d, 1.f / 120.f);
  s = fmaf(s, d, 1.f / 24.f);
  s = fmaf(s, d, 1.f / 6.f);
  s = fmaf(s, d, 0.5f);
  const float k = d * d * s;
  e = d + k;
  return k;
}

// A counted row's gradient coefficient grad_scale w c / temperature, from its
// maximum and its sum.  Every warp of the row works it out from the same values
// by the same operations, with the log probability's rounding: warps that took
// the rounded one could fall on the other side of a clip bound than the warp that
// writes the row's loss (`warp_writes`, `writes` by this lane), and each wrote its own slope.
__device__ __forceinline__ float finish_row(const ftmoe_policy_args& a, const RowInputs& in, MaxSum run, float zy,
                                            float inv_t, bool warp_writes, bool writes) {
  if (!a.dlogits && !warp_writes) return 0.f;
  const LogProb logp = log_prob(zy, run.m, run.s, a.temperature, inv_t);
  const float r = expf(logp.minus(in.old)), A = in.adv;
  const float bounded = r < 1.f - a.clip_low ? 1.f - a.clip_low : r > 1.f + a.clip_high ? 1.f + a.clip_high : r;
  const bool clipped = r * A > bounded * A;  // false for NaN, which then reaches the loss and the gradient
  float row = -(clipped ? bounded * A : r * A), c = clipped ? 0.f : -(A * r);
  if (a.ref_logp && a.kl_coef != 0.f) {
    float e;
    row += a.kl_coef * kl_term(-logp.minus(in.ref), e);
    c -= a.kl_coef * e;
  }
  if (writes) {
    a.row_loss[in.n] = row;
    if (a.logp) a.logp[in.n] = logp.value();
  }
  return c * (a.grad_scale * in.w * inv_t);
}
__device__ __forceinline__ void write_uncounted(const ftmoe_policy_args& a, int64_t n) {
  a.row_loss[n] = 0.f;
  if (a.logp) a.logp[n] = 0.f;
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
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(at),
               "l"(pack2(v.m, v.s)), "r"(at_bar)
               : "memory");
}

// Takes the work of a cluster that has not been launched yet; its first CTA's
// index, or none, arrives in every CTA of this cluster.
__device__ __forceinline__ void ask_for_row(void* response, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 "
      "[%0], [%1];" ::"r"(smem_u32(response)),
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

// A warp's pieces of a row: [lo, hi), and the whole ones [wlo, whi).
template <typename T>
struct Part {
  Row<T> z;
  RowInputs in;
  int lo, hi, wlo, whi;

  __device__ __forceinline__ int count() const { return hi - lo; }
  __device__ __forceinline__ int chunks() const { return (hi - lo + kChunk - 1) / kChunk; }
  // Chunk j as whole pieces [chunk_lo, chunk_hi); empty if they do not ascend.
  __device__ __forceinline__ int chunk_lo(int j) const { return max(wlo, lo + j * kChunk); }
  __device__ __forceinline__ int chunk_hi(int j) const { return min(whi, lo + (j + 1) * kChunk); }
};

// Waits that ran out: for a chunk (the warp's rows come out as NaN from then on,
// and it asks for no further chunk), and for the cluster (the warp leaves).
constexpr uint32_t kNoChunk = 1u << 30, kNoCluster = 1u << 31, kFailed = kNoChunk | kNoCluster;

// The limits of the waits, and whether a test withholds a chunk, so that one runs out.
struct Waits {
  uint64_t limit_ns, meeting_ns;
  int withhold;
};

// Gave up: waits (as long at most) for the copies that may still be on their way
// (the lane that fetches), and for what peers may have sent.  Apart from the
// kernels, whose loops it would cost registers (2% at N=4096 V=131072).
__device__ __noinline__ void settle(uint64_t* bar, uint32_t phases, bool fetches, uint64_t limit_ns, uint32_t* status) {
  if (!fetches) return;
  for (uint32_t left = phases << 2 >> 18; left; left &= left - 1) {
    const int j = __ffs(left) - 1;
    if (!mbar_wait(bar + j, phases >> j & 1, status, limit_ns)) break;
  }
}
__device__ __noinline__ void settle_cluster(uint64_t* meet, uint64_t* ask, uint32_t round, uint64_t limit_ns,
                                            uint32_t* status) {
  for (uint32_t r = round - 1; r <= round; ++r) {
    mbar_wait(meet + (r & 1), r >> 1 & 1, status, limit_ns);
    if (ask) mbar_wait(ask + (r & 1), r >> 1 & 1, status, limit_ns);
  }
}

// One warp's work on its part of a row, in its own shared memory.
template <typename T>
struct Worker {
  static constexpr int N = Row<T>::N;
  const ftmoe_policy_args& a;
  const int lane;
  uint32_t* const status;
  const float inv_t, k2;
  Pack<T, N>* buf;      // the part
  uint64_t* bar;        // a barrier for each chunk
  const Waits& waits;
  uint32_t phases = 0;  // of the barriers; from bit 16 on, chunks on their way (of the lane that fetches)

  __device__ Worker(const ftmoe_policy_args& args, int lane_, uint32_t* status_, Pack<T, N>* buf_, uint64_t* bar_,
                    const Waits& waits_)
      : a(args), lane(lane_), status(status_), inv_t(1.f / args.temperature), k2(kLog2e / args.temperature), buf(buf_),
        bar(bar_), waits(waits_) {}
  __device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity) const {
    return mbar_wait(b, parity, status, waits.limit_ns);
  }
  __device__ __forceinline__ T* vals() const { return reinterpret_cast<T*>(buf); }

  // The part of row n that is number `index` of 2^log2_parts * per_cta parts (CTA by CTA).
  __device__ __forceinline__ Part<T> part_of(int64_t n, int log2_ctas, int cta, int per_cta, int index) const {
    Part<T> p{Row<T>(static_cast<const T*>(a.logits) + n * a.ld, (int)a.V), row_inputs(a, n), 0, 0, 0, 0};
    const int pieces = p.z.pieces(), per = (pieces + (1 << log2_ctas) - 1) >> log2_ctas;
    const int each = (per + per_cta - 1) / per_cta, end = min(pieces, (cta + 1) * per);
    p.lo = min(end, cta * per + index * each);
    p.hi = min(end, p.lo + each);
    p.wlo = max(p.lo, (p.z.skip + N - 1) / N);
    p.whi = max(p.wlo, min(p.hi, p.z.end / N));
    return p;
  }
  // f(e) for the values e of the pieces that are not whole, among the part's pieces [begin, end).
  template <typename F>
  __device__ __forceinline__ void edges(const Part<T>& p, int begin, int end, F f) const {
    if (lane >= N) return;
    for (int i = p.lo + begin; i < min(p.wlo, p.lo + end); ++i) f(i * N + lane);
    for (int i = max(p.whi, p.lo + begin); i < p.lo + end; ++i) f(i * N + lane);
  }
  // Asks for a chunk's whole pieces (one lane; none where this warp has given
  // up, as the barrier may still wait for the row before).
  __device__ __forceinline__ void fetch(const Part<T>& p, int j) {
    const int from = p.chunk_lo(j), to = p.chunk_hi(j);
    if (p.in.w == 0.f || from >= to || (phases & kFailed)) return;
    phases |= 0x10000u << j;
    mbar_arrive_expect_tx(bar + j, (uint32_t)(to - from) * 16);
    bulk_g2s(buf + (from - p.lo), p.z.at + (int64_t)from * N, (uint32_t)(to - from) * 16, bar + j);
  }
  // The part's maximum and sum, this lane's; `summed(j)` after each chunk.
  template <typename F>
  __device__ __forceinline__ MaxSum sum(const Part<T>& p, F summed) {
    MaxSum r{-FLT_MAX, 0.f};
    if (p.wlo > p.lo || p.whi < p.hi) {
      edges(p, 0, p.count(), [&](int e) {
        vals()[e - p.lo * N] = e >= p.z.skip && e < p.z.end ? p.z.at[e] : from_f32<T>(-INFINITY);
      });
      fence_async_smem();
      __syncwarp();
    }
    for (int j = 0; j < p.chunks(); ++j) {
      if (p.chunk_lo(j) < p.chunk_hi(j)) {
        if (!(phases & kFailed) && wait(bar + j, phases >> j & 1)) {
          phases ^= 0x10001u << j;
        } else {
          phases |= kNoChunk;
        }
      }
      const int end = min(p.count(), (j + 1) * kChunk);
      int i = j * kChunk + lane;
      for (; i + 32 * (kUnroll - 1) < end; i += 32 * kUnroll) add_pieces<T, kUnroll>(buf + i, k2, r.m, r.s);
      for (; i < end; i += 32) add_pieces<T, 1>(buf + i, k2, r.m, r.s);
      summed(j);
    }
    if (phases & kFailed) r.s = NAN;
    return r;
  }
  // The part's gradient c (onehot - softmax), softmax z = 2^((x - m) k2 - ls),
  // in place and from there to dlogits; `left(j)` (one lane) once the copies up to
  // chunk j are under way.
  template <typename F>
  __device__ __forceinline__ void gradient(const Part<T>& p, float m, float ls, float c, float zy, F left) const {
    const Row<T> g(static_cast<T*>(a.dlogits) + p.in.n * a.ld_d, (int)a.V);
    const bool same = g.skip == p.z.skip;
    T* out = g.at + (g.skip - p.z.skip);  // out[e] belongs to the logit z.at[e]
    const int e0 = max(p.z.skip, p.lo * N), e1 = (int)min((int64_t)p.z.end, (int64_t)p.hi * N);
    auto mine = [&](int e) { return e >= p.z.skip && e < p.z.end; };
    if (c == 0.f) {  // nothing of the row's softmax is needed
      if (same) {
        for (int i = p.wlo + lane; i < p.whi; i += 32) store_pack<T, N>(out + (int64_t)i * N, zero_pack<T, N>());
        edges(p, 0, p.count(), [&](int e) {
          if (mine(e)) out[e] = from_f32<T>(0.f);
        });
      } else {
        for (int e = e0 + lane; e < e1; e += 32) out[e] = from_f32<T>(0.f);
      }
      return;
    }
    const int target = p.z.skip + (int)p.in.y - p.lo * N;  // among the part's values
    const float of_target = c * (1.f - exp2_fast((zy - m) * k2 - ls));
    for (int j = 0; j < p.chunks(); ++j) {
      const int begin = j * kChunk, end = min(p.count(), begin + kChunk);
      int i = begin + lane;
      for (; i + 32 * (kUnroll - 1) < end; i += 32 * kUnroll) gradient_of_pieces<T, kUnroll>(buf + i, k2, m, ls, c);
      for (; i < end; i += 32) gradient_of_pieces<T, 1>(buf + i, k2, m, ls, c);
      // the target's own term, by the lane that wrote its piece
      if (target >= begin * N && target < end * N && target / N % 32 == lane) vals()[target] = from_f32<T>(of_target);
      fence_async_smem();
      __syncwarp();
      if (!same) continue;
      edges(p, begin, end, [&](int e) {
        if (mine(e)) out[e] = vals()[e - p.lo * N];
      });
      if (lane == 0) {
        const int from = p.chunk_lo(j), to = p.chunk_hi(j);
        if (from < to) bulk_s2g(out + (int64_t)from * N, buf + (from - p.lo), (uint32_t)(to - from) * 16);
        bulk_commit();  // one group a chunk, empty or not
        left(j);
      }
    }
    if (!same) {  // dlogits' rows are of another alignment: value by value
      for (int e = e0 + lane; e < e1; e += 32) out[e] = vals()[e - p.lo * N];
    }
  }
};

// Long rows: the warps of a cluster of CTAs take a row.  Each warp copies its
// part of the row into its own shared memory, sums it, and after the warps have
// exchanged their maxima and sums, turns it into the gradient in place and
// sends that off: a row is read once and written once, no register holds a
// load in flight, and the warps meet once a row.  The copies go in chunks: a
// chunk is summed while later ones are on their way, and as soon as its
// gradient has left its buffer (without a gradient: as soon as it is summed)
// the next row's chunk is asked for.  Clusters take further rows from those not
// launched yet, so rows of weight 0, which cost half or nothing, leave no SM
// idle.  Memory bounds it: N=4096 V=131072 bf16, a fifth of the rows left out,
// 298 us, 95% of the copy rate; all rows 330 us.
template <typename T, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, kMinWarps / WARPS)
    k_policy(ftmoe_policy_args a, int part_pieces, int further, Waits waits, uint32_t* status) {
  extern __shared__ __align__(128) unsigned char policy_smem[];
  __shared__ uint64_t bars[WARPS][kMaxChunks];
  __shared__ uint64_t meet[2], ask[2];
  __shared__ __align__(16) uint4 response[2];
  __shared__ MaxSum exchange[2][kMaxRanks * WARPS];
  constexpr int N = Row<T>::N;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), log2_ranks = 31 - __clz(ranks);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool speaks = rank == 0 && threadIdx.x == 0;
  Worker<T> w(a, lane, status, reinterpret_cast<Pack<T, N>*>(policy_smem) + warp * part_pieces, bars[warp], waits);
  if (lane < kMaxChunks) mbar_init(bars[warp] + lane, 1);
  if (threadIdx.x < 2) {
    mbar_init(meet + threadIdx.x, 1);
    mbar_init(ask + threadIdx.x, 1);
  }
  fence_mbar_init();
  __syncwarp();
  uint32_t round = 0;  // rows met so far: slot and phase of what the cluster shares
  auto part_of = [&](int64_t n) { return w.part_of(n, log2_ranks, rank, WARPS, warp); };

  bool more = true;
  Part<T> p = part_of(blockIdx.x >> log2_ranks);  // the grid has no more clusters than rows
  check_target(a, p.in, speaks, status);
  if (lane == 0)  // the test withholds the first chunk of one warp
    for (int j = waits.withhold && blockIdx.x == 0 && warp == WARPS - 1; j < p.chunks(); ++j) w.fetch(p, j);
  cluster.sync();  // every CTA's barriers are set before a peer uses them
  // Thread 0 of each CTA: the number of a further row, into a slot.  With a
  // gradient the next row is needed late in a row, and asked for at its start
  // (a cluster that holds rows it cannot start yet is late at the end); without
  // one it is needed at the start, and asked for a row ahead.
  auto ask_into = [&](uint32_t slot) {
    mbar_arrive_expect_tx(ask + slot, 16);
    if (rank == 0) ask_for_row(response + slot, ask + slot);
  };
  if (!a.dlogits && further && threadIdx.x == 0) ask_into(0);
  while (more) {
    const uint32_t slot = round & 1, turn = round >> 1 & 1;
    if (threadIdx.x == 0) {
      mbar_arrive_expect_tx(meet + slot, (uint32_t)(ranks * WARPS * sizeof(MaxSum)));
      if (a.dlogits && further) ask_into(slot);
    }
    // The next row: its number, and its inputs on their way.
    Part<T> next = p;
    int next_chunks = 0, asked = 0;  // the next row's chunks, and those asked for
    auto find_next = [&]() {
      more = false;
      if (!further) return;
      uint32_t cta = 0;
      if (w.wait(ask + slot, turn)) more = row_given(response + slot, cta);
      else w.phases |= kNoCluster;
      fence_async_smem();  // read before the slot is given again
      if (more) next = part_of(cta >> log2_ranks);
    };
    auto check_next = [&]() {
      if (!more) return;
      check_target(a, next.in, speaks, status);
      next_chunks = next.chunks();
    };
    if (!a.dlogits) {
      find_next();
      if (more && threadIdx.x == 0) ask_into(slot ^ 1);
      check_next();
    }
    MaxSum run{-FLT_MAX, 0.f};
    float zy = 0.f;
    if (p.in.w != 0.f) {
      zy = to_f32(p.z.at[p.z.skip + p.in.y]);
      run = w.sum(p, [&](int) {
        if (a.dlogits) return;
        __syncwarp();
        if (lane == 0 && asked < next_chunks) w.fetch(next, asked++);
      });
      // zy is in hand before the warps meet: dlogits may be the logits themselves
      if (isnan(zy)) run.s = NAN;
    }
    if (a.dlogits) find_next();

    // Every warp tells every CTA.  Two sets of slots suffice: a warp sends
    // into a set again two rows on, when it has heard in the next row from
    // every warp of the cluster, each after its reads here.
    // A wait that ran out makes the row's sum NaN, here and in every CTA that hears
    // of it; the wait for the others is longer than those before it together.
    static_assert(kMaxRanks * WARPS <= 32, "a lane a sender");
    if (w.phases & kFailed) run.s = NAN;
    run = warp_join(run, w.k2);
    if (lane < ranks) send(run, &exchange[slot][rank * WARPS + warp], meet + slot, lane);
    if (!mbar_wait(meet + slot, turn, status, waits.meeting_ns)) w.phases |= kNoCluster;
    run = lane < ranks * WARPS ? exchange[slot][lane] : MaxSum{-FLT_MAX, 0.f};
    if (w.phases & kFailed) run.s = NAN;
    run = warp_join(run, w.k2);
    if (isnan(run.s)) {
      w.phases |= __reduce_or_sync(0xffffffffu, w.phases) & kFailed;
      if (w.phases & kNoCluster) more = false;
    }
    ++round;
    float c = 0.f;
    const float log2_s = log2f(run.s);
    if (p.in.w != 0.f) c = finish_row(a, p.in, run, zy, w.inv_t, rank == 0 && warp == 0, speaks);
    else if (speaks) write_uncounted(a, p.in.n);
    if (a.dlogits) {
      check_next();
      if (c == 0.f) {  // the buffer is free
        __syncwarp();
        if (lane == 0)
          for (; asked < next_chunks; ++asked) w.fetch(next, asked);
        asked = next_chunks;
      }
      w.gradient(p, run.m, log2_s, c, zy, [&](int j) {
        if (j < kLag) return;
        bulk_wait_read<kLag>();  // the gradient of chunk j - kLag has left its buffer
        if (asked < next_chunks) w.fetch(next, asked++);
      });
    }
    __syncwarp();
    if (lane == 0) {
      bulk_wait_read<0>();
      for (; asked < next_chunks; ++asked) w.fetch(next, asked);
    }
    p = next;
  }
  pdl_launch_dependents();
  if (lane == 0) bulk_wait_read<0>();
  // No CTA leaves before every message and question of the cluster is on its way
  // (each wait before has its limit), nor, if a wait ran out, before what may still
  // come to it has come or had the limit's time once more.
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (!(w.phases & kFailed)) return;
  settle(bars[warp], w.phases, lane == 0, waits.limit_ns, status);
  if (w.phases & kNoCluster) settle_cluster(meet, further ? ask : nullptr, round, waits.limit_ns, status);
}

// Short rows: a warp takes a row, and has the next one on its way in a second
// buffer while it turns one into its gradient.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, kMinWarps / kWarps)
    k_policy_short(ftmoe_policy_args a, int pieces, Waits waits, uint32_t* status) {
  extern __shared__ __align__(128) unsigned char policy_smem[];
  __shared__ uint64_t bars[2][kWarps][kShortChunks];
  constexpr int N = Row<T>::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pack<T, N>* first = reinterpret_cast<Pack<T, N>*>(policy_smem) + warp * 2 * pieces;
  Worker<T> w(a, lane, status, first, bars[0][warp], waits);
  if (lane < 2 * kShortChunks) mbar_init(bars[lane / kShortChunks][warp] + lane % kShortChunks, 1);
  fence_mbar_init();
  __syncwarp();
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t n = (int64_t)blockIdx.x * kWarps + warp;
  if (n >= a.N) return;
  // The buffer in use is w's; the other one's barriers have other phases.
  int side = 0;
  uint32_t other_phases = 0;
  auto turn = [&]() {
    side ^= 1;
    w.buf = first + side * pieces;
    w.bar = bars[side][warp];
    const uint32_t t = w.phases;
    w.phases = other_phases;
    other_phases = t;
  };
  auto fetch_row = [&](const Part<T>& p, int j) {  // one lane
    for (; j < p.chunks(); ++j) w.fetch(p, j);
  };
  Part<T> p = w.part_of(n, 0, 0, 1, 0);
  check_target(a, p.in, lane == 0, status);
  // the test withholds one warp's first chunk
  if (lane == 0) fetch_row(p, waits.withhold && blockIdx.x == 0 && warp == 0);
  bool more = true;
  while (more) {  // once a wait has run out, the warp's rows come out as NaN, and none is asked for
    n += step;
    more = n < a.N;
    Part<T> next = p;
    if (more) next = w.part_of(n, 0, 0, 1, 0);
    MaxSum run{-FLT_MAX, 0.f};
    float zy = 0.f, c = 0.f;
    if (p.in.w != 0.f) {
      zy = to_f32(p.z.at[p.z.skip + p.in.y]);
      run = w.sum(p, [](int) {});
    }
    if (more) {
      check_target(a, next.in, lane == 0, status);
      turn();
      if (lane == 0) {
        bulk_wait_read<0>();  // the other buffer's gradient has left
        fetch_row(next, 0);
      }
      turn();
    }
    float log2_s = 0.f;
    if (p.in.w != 0.f) {
      run = warp_join(run, w.k2);
      log2_s = log2f(run.s);
      c = finish_row(a, p.in, run, zy, w.inv_t, true, lane == 0);
    } else if (lane == 0) {
      write_uncounted(a, p.in.n);
    }
    if (a.dlogits) w.gradient(p, run.m, log2_s, c, zy, [](int) {});
    p = next;
    turn();
  }
  if (lane == 0) bulk_wait_read<0>();
  if (!(w.phases & kFailed) || lane != 0) return;  // (a lane that fetched and waited in time has nothing on its way)
  for (int s = 0; s < 2; ++s, turn()) settle(w.bar, w.phases, true, waits.limit_ns, status);
}

// Rows too long for a cluster's shared memory (8 parts of 216 KB): the logits are
// read a second time.  256 rows of 2^20 values, all with a gradient: fp32 628 us,
// 5.1 TB/s of three moves; bf16 411 us, 3.9 TB/s, where a piece holds twice the
// exponentials.
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
    RowInputs in = row_inputs(a, n);
    check_target(a, in, rank == 0 && tid == 0, status);
    const Row<T> z(static_cast<const T*>(a.logits) + n * a.ld, (int)a.V);
    const int per = (z.pieces() + ranks - 1) / ranks, lo = min(z.pieces(), rank * per), hi = min(z.pieces(), lo + per);
    float c = 0.f, ls = 0.f, m = 0.f;
    if (in.w != 0.f) {
      const float zy = to_f32(z.at[z.skip + in.y]);
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
      c = finish_row(a, in, run, zy, 1.f / a.temperature, rank == 0 && warp == 0, rank == 0 && tid == 0);
    } else if (rank == 0 && tid == 0) {
      write_uncounted(a, n);
    }
    if (!a.dlogits) continue;
    const Row<T> g(static_cast<T*>(a.dlogits) + n * a.ld_d, (int)a.V);
    const bool same = g.skip == z.skip;
    Row<T> out = g;  // at the logits' pieces; of another alignment: written value by value
    out.at += g.skip - z.skip;
    out.skip = z.skip;
    out.end = z.end;
    const int target = z.skip + (int)in.y;
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

// loss = sum_n w_n row_n in a fixed order, by one CTA: in fp32 with each
// addition's rounding kept and added at the end (FP64, of which an SM does two
// a cycle, took 9 us of 16384 rows).
struct Sum2 {
  float s, e;
  __device__ __forceinline__ void add(float v) {
    const float t = __fadd_rn(s, v), u = __fsub_rn(t, s);
    e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, u)), __fsub_rn(v, u)));
    s = t;
  }
};
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads)
    k_policy_sum(const float* weight, const float* row_loss, int64_t N, float* loss) {
  __shared__ Sum2 part[kSumThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  Sum2 t{0.f, 0.f};
  const float each = 1.f / (float)N;
  for (int64_t n0 = threadIdx.x; n0 < N; n0 += 8 * kSumThreads) {
    float v[8], w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t n = min(n0 + u * kSumThreads, N - 1);
      v[u] = row_loss[n];
      w[u] = weight ? weight[n] : each;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (n0 + u * kSumThreads >= N) break;
      const float r = __fmul_rn(v[u], w[u]);
      t.add(r);
      t.e = __fadd_rn(t.e, __fmaf_rn(v[u], w[u], -r));
    }
  }
  auto join = [&](int width) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= width) continue;
      const float s = __shfl_down_sync(0xffffffffu, t.s, o), e = __shfl_down_sync(0xffffffffu, t.e, o);
      t.add(s);
      t.e = __fadd_rn(t.e, e);
    }
  };
  join(32);
  if (lane == 0) part[warp] = t;
  __syncthreads();
  if (warp == 0) {
    t = part[lane];
    join(32);
    // NaN and infinities are the sum's own: their rounding terms say nothing
    if (lane == 0) *loss = isfinite(t.s) ? t.s + t.e : t.s;
  }
}

// A CTA's shared memory for its part of a row, at most; what an SM has for all of them.
constexpr int kStageMax = 216 * 1024, kSmemSm = 226 * 1024;
// Of a CTA and of each warp besides: the system's own, barriers, slots.
constexpr int kFixedSmem = 1280, kWarpSmem = 288;
// Rows up to kShortBytes may be a warp's: 16384 bf16 rows of 4 KB take 35 us so and
// 64 us as two warps', of 16 KB 172 and 111 us.  Up to kShortAlways they are even
// where that leaves warps idle.
constexpr int kShortBytes = 8 * 1024, kShortAlways = 2 * 1024;
// Rows up to here are two warps' instead of four's: 16384 rows of 16 KB take 111 and
// 117 us, 8192 of 24 KB 79 and 83 us, of 32 KB 106 and 96 us.
constexpr int kTwoWarpBytes = 24 * 1024;

}  // namespace

static_assert(kShortBytes / 16 <= kShortChunks * kChunk && 2 * kShortChunks <= 32,
              "a short row's chunks have barriers");
static_assert(kStageMax / 16 / kWarps <= kMaxChunks * kChunk && kMaxChunks <= 14,
              "a part's chunks have barriers and phases");

cudaError_t policy_set_limits() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto type) {
    using T = decltype(type);
    for (const void* k :
         {(const void*)k_policy_short<T>, (const void*)k_policy<T, 2>, (const void*)k_policy<T, kWarps>}) {
      const cudaError_t r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMax);
      if (r != cudaSuccess) return r;
    }
    return cudaSuccess;
  };
  for (int t : {FTMOE_BF16, FTMOE_FP32, FTMOE_FP16})
    if ((e = with_dtype(t, set)) != cudaSuccess) return e;
  return e;
}

cudaError_t launch_policy_loss(const TrainDevice& d, const ftmoe_policy_args& a, cudaStream_t s) {
  if (a.N > 0) {
    const int64_t pieces = (a.V * dtype_bytes(a.dtype) + 15 + 14) / 16;  // of a row at any alignment, at most
    const int64_t bytes = pieces * 16;
    const bool many = a.N >= 8 * d.num_sms;
    const bool is_short = bytes <= kShortBytes && (bytes <= kShortAlways || many);
    const int warps = !is_short && many && bytes <= kTwoWarpBytes ? 2 : kWarps;
    auto part = [&](int ranks) { return ((pieces + ranks - 1) / ranks + warps - 1) / warps; };  // a warp's pieces
    auto cta_bytes = [&](int ranks) { return part(ranks) * warps * 16; };
    auto resident = [&](int64_t smem) {
      return std::min<int64_t>(kMinWarps / warps, kSmemSm / (smem + kFixedSmem + warps * kWarpSmem));
    };
    // The ranks that have most of an SM's shared memory in use; of (nearly) equals,
    // the most, whose CTAs are more.
    int ranks = 1;
    for (int r = 2; r <= kMaxRanks && warps == kWarps; r *= 2)
      if (cta_bytes(r) * resident(cta_bytes(r)) >= cta_bytes(ranks) * resident(cta_bytes(ranks)) * 98 / 100) ranks = r;
    // few rows: spread each over more CTAs while the SMs are not full and a part has work for its warps
    while (ranks < kMaxRanks && a.N * ranks < 2 * d.num_sms && cta_bytes(ranks) >= 8192) ranks *= 2;
    if (cta_bytes(ranks) > kStageMax) ranks = kMaxRanks;
    const int64_t smem = is_short ? pieces * 2 * kWarps * 16 : cta_bytes(ranks);
    // a part has a barrier for each chunk, so it has kMaxChunks of them at most
    const bool staged = smem <= kStageMax && (is_short || part(ranks) <= kMaxChunks * kChunk);
    if (is_short) ranks = 1;
    cudaLaunchConfig_t c{};
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 1;
    c.blockDim = dim3(staged ? warps * 32 : kLongThreads);
    c.dynamicSmemBytes = staged ? (size_t)smem : 0;
    const int64_t want = is_short ? (a.N + kWarps - 1) / kWarps : a.N;
    // short rows: as many warps as fit; long ones: a cluster a row, of which those that
    // run take the rest over (memory ends before the grid does)
    const int64_t room = is_short ? d.num_sms * resident(smem) : staged ? INT32_MAX / ranks : 1 << 24;
    c.gridDim = dim3((unsigned)(std::min(want, room) * ranks));
    const int further = a.N * ranks > d.num_sms;  // else no cluster waits to be launched
    const uint64_t limit_ns = d.test_wait_ns ? d.test_wait_ns : kWaitLimitNs;
    const Waits waits{limit_ns, 4 * limit_ns, d.test_wait_ns != 0};
    cudaError_t e = with_dtype(a.dtype, [&](auto type) {
      using T = decltype(type);
      if (!staged) return cudaLaunchKernelEx(&c, k_policy_long<T>, a, d.status);
      if (is_short) return cudaLaunchKernelEx(&c, k_policy_short<T>, a, (int)pieces, waits, d.status);
      const auto k = warps == 2 ? k_policy<T, 2> : k_policy<T, kWarps>;
      return cudaLaunchKernelEx(&c, k, a, (int)part(ranks), further, waits, d.status);
    });
    if (e != cudaSuccess) return e;
  }
  return launch_after(k_policy_sum, 1, kSumThreads, s, a.weight, a.row_loss, a.N, a.loss);
}

}  // namespace ftmoe
