// Gated linear recurrence (gconv_gated_scan_fwd / _bwd).
//
//   l_t = -c softplus(lam) sig(r_t),  a_t = exp(l_t)
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sig(i_t) x_t
//
// Each channel of each sequence is its own recurrence.
#include <initializer_list>
#include <type_traits>

#include "seq.h"
#include "seq_vec.cuh"

namespace gconv {
namespace {

constexpr int kChunk = GCONV_SCAN_CHUNK;

__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Logistic function, a few units in the last place of fp32: 0 and 1 at the
// infinities, NaN for NaN, 0 below exp(-87).
__device__ __forceinline__ float sigmoid(float v) { return rcp_approx(1.f + __expf(-v)); }

// rate = c * softplus(lam): once for each channel.  Finite, so that a gate of 0,
// which stands for a row past the sequence's end, leaves the state as it is: an
// infinite rate times it would be NaN.  (exp is 0 from a rate of 104 on.)
__device__ __forceinline__ float decay_rate(float lam, float c) {
  const float rate = c * (lam > 0.f ? lam + log1pf(expf(-lam)) : log1pf(expf(lam)));
  return rate > 3.4e38f ? 3.4e38f : rate;  // NaN stays
}

// exp(l) - 1 for -kSmall <= l <= 0: the Taylor polynomial, which loses nothing
// to the subtraction (its first dropped term is below 2^-25 of the result).
constexpr float kSmall = 0.35f;
__device__ __forceinline__ float expm1_small(float l) {
  float p = fmaf(l, 1.f / 5040.f, 1.f / 720.f);
  p = fmaf(l, p, 1.f / 120.f);
  p = fmaf(l, p, 1.f / 24.f);
  p = fmaf(l, p, 1.f / 6.f);
  p = fmaf(l, p, 0.5f);
  p = fmaf(l, p, 1.f);
  return l * p;
}

// sig(v) and 1 - sig(v), neither as a difference from 1.
__device__ __forceinline__ void sigmoid_pair(float v, float& sig, float& rest) {
  const float t = __expf(-fabsf(v)), w = __fdividef(1.f, 1.f + t);
  sig = v >= 0.f ? w : t * w;
  rest = v >= 0.f ? t * w : w;
}

// What the decay gate's value v gives: g = sig(v) and o = 1 - g, a = exp(-rate g),
// s = sqrt(1 - a^2) and k = g / s (0 where s is 0), the factor that the
// gradient of s needs.  1 - a^2 = -e (2 + e) with e = a - 1.
struct Gate {
  float g, o, a, s, k;
};
// Channels by their rate.  Slow ones have |l| <= kSmall throughout.  With those
// and plain ones, and ordinary gates (v >= kFastGate), nothing comes near the
// smallest or the largest number.  8 x 2048 x 2048 bf16, forward / backward: slow
// 71 / 104 us, plain 77 / 110, steep 78 / 110, any 195 / 205.
constexpr float kFastGate = -60.f, kFastInput = -25.f;  // D q stays below 2^127
// Steep ones are plain where the gates are ordinary: below exp(-87), where the packed
// arithmetic takes a gate as 0, their sqrt(1 - a^2), sqrt(2 rate sig(r)), is
// not yet below 1e-18.
enum RateKind { kRateAny = 0, kRateSteep = 1, kRatePlain = 2, kRateSlow = 3 };
constexpr float kSteep = 32.f;
__device__ __forceinline__ RateKind rate_kind(float rate) {
  if (!(rate >= 1e-9f && rate <= 1e30f)) return kRateAny;
  return rate <= kSmall ? kRateSlow : rate <= kSteep ? kRatePlain : kRateSteep;
}
// The kind that holds for all channels of a warp.
template <int V>
__device__ __forceinline__ RateKind warp_kind(const float (&rate)[V]) {
  int k = kRateSlow;
#pragma unroll
  for (int v = 0; v < V; ++v) k = min(k, (int)rate_kind(rate[v]));
  return (RateKind)__reduce_min_sync(0xffffffffu, k);
}
// Any channel and gate.  Far from 0, a comes from exp itself (1 + e would lose
// a small a).  For a gate below exp(-40), where 1 - a^2 = 2 rate sig(v) is below 1e-8, s
// and k come from that by sig(v) = exp(v / 2)^2, because sig(v) and l themselves may be
// subnormal.
__device__ __forceinline__ Gate gate_any(float v, float rate) {
  Gate q;
  sigmoid_pair(v, q.g, q.o);
  const float l = -rate * q.g;
  const bool near = l > -kSmall;
  const float e0 = expm1_small(l), a0 = __expf(l);
  const float e = near ? e0 : a0 - 1.f;
  q.a = near ? 1.f + e0 : a0;
  const float z = fmaf(-e, e, -2.f * e);
  q.s = sqrtf(z);
  q.k = z > 0.f ? q.g / q.s : 0.f;
  if (v < -40.f) {
    const float half = expf(0.5f * v), root = 1.41421356f * sqrtf(rate);
    if (half * root < 1e-4f) {
      q.s = half * root;
      q.k = root > 0.f ? half / root : 0.f;
    }
  }
  return q;
}

// ---------------------------------------------------------------------------
// One token: a thread for each channel of each sequence.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs s) {
  allow_dependent_launch();
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (id >= s.B * s.D) return;
  const int64_t b = s.B == 1 ? 0 : id / s.D;
  const int d = (int)(id - b * s.D);
  grid_dependency_wait();
  float h = s.h0 ? s.h0[id] : 0.f;
  if (s.saved) s.saved[id] = h;
  float out = 0.f;
  if (seq_len(s.lens, b, 1) == 1) {
    const Gate q = gate_any(Elem<T>::to_f32(static_cast<const T*>(s.r)[b * s.sr.b + d]), decay_rate(s.lam[d], s.decay));
    h = fmaf(q.a, h, q.s * sigmoid(Elem<T>::to_f32(static_cast<const T*>(s.i)[b * s.si.b + d])) *
                         Elem<T>::to_f32(static_cast<const T*>(s.x)[b * s.sx.b + d]));
    out = h;
  }
  static_cast<T*>(s.y)[b * s.sy.b + d] = Elem<T>::from_f32(out);
  if (s.hT) s.hT[id] = h;
}

// ---------------------------------------------------------------------------
// The scan over time.  A block owns a slab of 32 V channels of one sequence
// and walks its tokens in tiles of W segments of S; warp w takes segment w of a
// tile, lane l the channels l V ... l V + V - 1, so a row of a slab is one
// 128-byte line of 16-bit or 32-bit values.
//
// A segment is the map h -> P h + H.  Each warp runs its S steps from H = 0
// and P = 1 and keeps every (P_s, H_s) in registers; the warps exchange their
// segments' maps through shared memory, fold the ones before their own onto
// the carried state, and finish with y_s = H_s + P_s h.  Inputs are read once.
// The next tile's rows are already on their way while a tile is exchanged.
//
// Where there are too few slabs to fill the GPU, a cluster of ns blocks shares
// one: block k of the cluster takes tiles k, ns + k, ...  The blocks' maps
// travel through distributed shared memory, counted by a barrier in each block.
// ---------------------------------------------------------------------------
constexpr int kMaxSplit = 12;  // blocks in a cluster (see split_of)

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The end of a block: none of a cluster leaves while another may send to it
// (only after a wait that ran out could one be so far ahead).
template <bool CL>
__device__ __forceinline__ void leave() {
  if constexpr (CL) {
    cluster_arrive();
    cluster_wait();
  }
}

// A map h -> p h + q for the V channels of a lane, as one word of shared memory.
template <int V> struct Map;
template <> struct alignas(16) Map<2> {
  float p[2], q[2];
};
template <> struct alignas(8) Map<1> {
  float p[1], q[1];
};
// Sends m to the place of `at` in the shared memory of block `rank` of the
// cluster, and its bytes to the count of that block's barrier `bar`.  (A cluster
// barrier would have to order the rows of y that are still being written.)
__device__ __forceinline__ void send_map(Map<2>* at, uint64_t* bar, int rank, const Map<2>& m) {
  uint32_t to, done;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(done) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
               "f"(m.p[0]), "f"(m.p[1]), "f"(m.q[0]), "f"(m.q[1]), "r"(done)
               : "memory");
}
__device__ __forceinline__ void send_map(Map<1>* at, uint64_t* bar, int rank, const Map<1>& m) {
  uint32_t to, done;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(done) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
               "f"(m.p[0]), "f"(m.q[0]), "r"(done)
               : "memory");
}
// c = m(c)
__device__ __forceinline__ void apply(const Map<1>& m, float (&c)[1]) { c[0] = fmaf(m.p[0], c[0], m.q[0]); }
__device__ __forceinline__ void apply(const Map<2>& m, float (&c)[2]) {
  const F2 r = fma2(f2(m.p[0], m.p[1]), f2(c[0], c[1]), f2(m.q[0], m.q[1]));
  c[0] = lo(r), c[1] = hi(r);
}
// c = m after c
__device__ __forceinline__ void compose(const Map<1>& m, Map<1>& c) {
  apply(m, c.q);
  c.p[0] *= m.p[0];
}
__device__ __forceinline__ void compose(const Map<2>& m, Map<2>& c) {
  apply(m, c.q);
  const F2 r = mul2(f2(m.p[0], m.p[1]), f2(c.p[0], c.p[1]));
  c.p[0] = lo(r), c.p[1] = hi(r);
}

// Maps of the segments of a block and of the blocks of a cluster.
template <int V, int W>
struct MapBuffers {
  Map<V> warp[2][W][32];
  Map<V> block[2][kMaxSplit][32];
  uint64_t bar[2];  // counts the bytes of block[k]
};

// What an exchange needs besides the maps themselves.
struct Place {
  int warp, lane, rank, ns;
  int* status;
  uint64_t limit;  // of a wait; 0 after one has run out: the walk then ends without waiting
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, int site) {
    if (mbar_wait(bar, parity, limit)) return;
    if (limit != 0) report(status, kDevTimeout, site);
    limit = 0;
  }
};
// Thread 0, before any other block may send: the barriers, each waiting for the
// maps of all ns blocks.
template <int V, int W>
__device__ __forceinline__ void init_maps(MapBuffers<V, W>& m, int ns) {
  for (int k = 0; k < 2; ++k) {
    mbar_init(&m.bar[k], 1);
    mbar_arrive_expect_tx(&m.bar[k], ns * 32 * (uint32_t)sizeof(Map<V>));
  }
  fence_mbar_init();
}

// The exchange of a round, in two halves so that work can lie between them.
// publish: this warp's map, the block's, and (in a cluster) its way to the other
// blocks.  collect: the carried value before this warp's segment; `carry` moves
// on to the value after the round.  Rounds alternate between two buffers: a
// block sends its maps of round k + 2 after it has collected round k + 1, for
// which every block had finished collecting round k.
// REV: the order is from the last block and warp to the first.
template <int V, int W, bool CL, bool REV>
__device__ __forceinline__ void publish(MapBuffers<V, W>& m, uint32_t round, const Place& at, const float (&p)[V],
                                        const float (&q)[V], Map<V>& before) {
  const int buf = (int)(round & 1);
  Map<V> own;
#pragma unroll
  for (int v = 0; v < V; ++v) own.p[v] = p[v], own.q[v] = q[v];
  m.warp[buf][at.warp][at.lane] = own;
  asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory");  // the W walking warps
  if constexpr (CL) {
    // the block has collected the round before: its barrier is free for the next one
    if (threadIdx.x == 0 && round > 0)
      mbar_arrive_expect_tx(&m.bar[buf ^ 1], at.ns * 32 * (uint32_t)sizeof(Map<V>));
    // The block's map first, as a tree, because others wait for it: warp w tells
    // block w (and w + W, ...) of the cluster.
    Map<V> o[W], tree[W];
#pragma unroll
    for (int k = 0; k < W; ++k) tree[k] = o[k] = m.warp[buf][REV ? W - 1 - k : k][at.lane];
#pragma unroll
    for (int w = 1; w < W; w *= 2)
#pragma unroll
      for (int k = 0; k + w < W; k += 2 * w) compose(tree[k + w], tree[k]);
    for (int to = at.warp; to < at.ns; to += W) send_map(&m.block[buf][at.rank][at.lane], &m.bar[buf], to, tree[0]);
    // the map before this warp
    const int place = REV ? W - 1 - at.warp : at.warp;
#pragma unroll
    for (int v = 0; v < V; ++v) before.p[v] = 1.f, before.q[v] = 0.f;
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      if (k < place) compose(o[k], before);
  }
}
template <int V, int W, bool CL, bool REV>
__device__ __forceinline__ void collect(MapBuffers<V, W>& m, uint32_t round, Place& at, const Map<V>& before,
                                        float (&carry)[V], float (&start)[V]) {
  const int buf = (int)(round & 1);
  if constexpr (!CL) {
    const int place = REV ? W - 1 - at.warp : at.warp;
#pragma unroll
    for (int v = 0; v < V; ++v) start[v] = carry[v];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      apply(m.warp[buf][REV ? W - 1 - k : k][at.lane], carry);
      if (k < place) {
#pragma unroll
        for (int v = 0; v < V; ++v) start[v] = carry[v];
      }
    }
  } else {
    at.wait(&m.bar[buf], (uint32_t)(round >> 1) & 1u, 71);
    const int rank = REV ? at.ns - 1 - at.rank : at.rank;
#pragma unroll
    for (int v = 0; v < V; ++v) start[v] = carry[v];
#pragma unroll
    for (int h = 0; h < kMaxSplit; h += 4) {  // four loads at a time
      if (h < at.ns) {
        Map<V> o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (h + k < at.ns) o[k] = m.block[buf][REV ? at.ns - 1 - h - k : h + k][at.lane];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (h + k < at.ns) apply(o[k], carry);
          if (h + k < rank) {
#pragma unroll
            for (int v = 0; v < V; ++v) start[v] = carry[v];
          }
        }
      }
    }
    apply(before, start);
  }
}
template <int V, int W, bool CL, bool REV>
__device__ __forceinline__ void exchange(MapBuffers<V, W>& m, uint32_t round, Place& at, const float (&p)[V],
                                         const float (&q)[V], float (&carry)[V], float (&start)[V]) {
  Map<V> before;
  publish<V, W, CL, REV>(m, round, at, p, q, before);
  collect<V, W, CL, REV>(m, round, at, before, carry, start);
}

// The smallest of the raw values (NaN is passed over).
__device__ __forceinline__ float lowest(float m, const Raw<float, 1>& r) { return fminf(m, __uint_as_float(r.w[0])); }
template <int V>
__device__ __forceinline__ __half2 lowest(__half2 m, const Raw<__half, V>& r) {
  const uint32_t w = V == 1 ? r.w[0] | r.w[0] << 16 : r.w[0];
  return __hmin2(m, *reinterpret_cast<const __half2*>(&w));
}
template <int V>
__device__ __forceinline__ __nv_bfloat162 lowest(__nv_bfloat162 m, const Raw<__nv_bfloat16, V>& r) {
  const uint32_t w = V == 1 ? r.w[0] | r.w[0] << 16 : r.w[0];
  return __hmin2(m, *reinterpret_cast<const __nv_bfloat162*>(&w));
}
template <typename T> struct Low;
template <> struct Low<float> {
  using type = float;
  static __device__ __forceinline__ float zero() { return 0.f; }
  static __device__ __forceinline__ float get(float m) { return m; }
};
template <> struct Low<__half> {
  using type = __half2;
  static __device__ __forceinline__ __half2 zero() { return __float2half2_rn(0.f); }
  static __device__ __forceinline__ float get(__half2 m) { return fminf(__low2float(m), __high2float(m)); }
};
template <> struct Low<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ __nv_bfloat162 zero() { return __float2bfloat162_rn(0.f); }
  static __device__ __forceinline__ float get(__nv_bfloat162 m) { return fminf(__low2float(m), __high2float(m)); }
};

// Whether all gates of a warp's segment are ordinary ones.
template <typename T, int V, int S>
__device__ __forceinline__ bool all_fast(const Raw<T, V> (&r)[S], const Raw<T, V> (&i)[S]) {
  typename Low<T>::type m = Low<T>::zero(), mi = Low<T>::zero();
#pragma unroll
  for (int k = 0; k < S; ++k) m = lowest(m, r[k]), mi = lowest(mi, i[k]);
  return __all_sync(0xffffffffu, Low<T>::get(m) >= kFastGate && Low<T>::get(mi) >= kFastInput);
}

// S rows of a tensor from token t, channels at p: those before n, zeros past it.
template <typename T, int V, int S>
__device__ __forceinline__ void ld_rows(Raw<T, V> (&out)[S], const T* p, int64_t stride, int64_t t, int64_t n, bool mine) {
  p += t * stride;
  if (mine && t + S <= n) {
#pragma unroll
    for (int k = 0; k < S; ++k) out[k] = ld_raw<T, V>(p + k * stride);
  } else {
#pragma unroll
    for (int k = 0; k < S; ++k) out[k] = mine && t + k < n ? ld_raw<T, V>(p + k * stride) : zero_raw<T, V>();
  }
}

__device__ __forceinline__ F2 rcp2(F2 a) { return f2(rcp_approx(lo(a)), rcp_approx(hi(a))); }
__device__ __forceinline__ F2 rsqrt2(F2 a) { return f2(rsqrt_approx(lo(a)), rsqrt_approx(hi(a))); }
__device__ __forceinline__ float ex2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The constants of the packed gate arithmetic.  Its instructions take
// registers only; made once by statements the compiler may not repeat, the
// pairs stay in registers over the walk.
struct GateConsts {
  F2 nlog2e, one, none, c6, c5, c4, c3, c2, c1, tiny, zero;
};
__device__ __forceinline__ F2 pinned(float v) {
  F2 r;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ GateConsts gate_consts() {
  return {pinned(-1.4426950408889634f), pinned(1.f),          pinned(-1.f),       pinned(1.f / 5040.f), pinned(-1.f / 720.f),
          pinned(1.f / 120.f),          pinned(-1.f / 24.f), pinned(1.f / 6.f), pinned(-0.5f),       pinned(1e-37f),
          pinned(0.f)};
}
// exp(-v), and 1 + exp(-v)
__device__ __forceinline__ F2 exp_neg2(const GateConsts& c, F2 v) {
  const F2 m = mul2(v, c.nlog2e);
  return f2(ex2_approx(lo(m)), ex2_approx(hi(m)));
}
__device__ __forceinline__ F2 one_plus_exp_neg2(const GateConsts& c, F2 v) { return add2(exp_neg2(c, v), c.one); }
// 1 - exp(-m) for 0 <= m <= kSmall: expm1_small for a pair, with the sign out.
__device__ __forceinline__ F2 one_minus_exp_neg2(const GateConsts& c, F2 m) {
  F2 p = fma2(m, c.c6, c.c5);
  p = fma2(m, p, c.c4);
  p = fma2(m, p, c.c3);
  p = fma2(m, p, c.c2);
  p = fma2(m, p, c.c1);
  p = fma2(m, p, c.one);
  return mul2(m, p);
}

// a = exp(-m) and e = 1 - a for a pair, m >= 0.  Plain channels: the polynomial
// up to kSmall, a from exp itself past it (1 - e would lose a small a).
template <RateKind K>
__device__ __forceinline__ void decay_pair(const GateConsts& c, F2 m, F2& e, F2& a) {
  e = one_minus_exp_neg2(c, m);
  a = fma2(e, c.none, c.one);
  if constexpr (K == kRatePlain) {
    const F2 t = mul2(m, c.nlog2e), far_a = f2(ex2_approx(lo(t)), ex2_approx(hi(t))), far_e = fma2(far_a, c.none, c.one);
    const bool l = lo(m) > kSmall, h = hi(m) > kSmall;
    e = f2(l ? lo(far_e) : lo(e), h ? hi(far_e) : hi(e));
    a = f2(l ? lo(far_a) : lo(a), h ? hi(far_a) : hi(a));
  }
}

// The pair `j` of a segment's values in the order (token, channel): the two
// channels of a token, or one channel of two tokens.
template <typename T, int V, int S>
__device__ __forceinline__ F2 pair_of(const Raw<T, V> (&r)[S], int j) {
  if constexpr (V == 2) {
    float f[2];
    widen<T, 2>(r[j], f);
    return f2(f[0], f[1]);
  } else {
    float a[1], b[1];
    widen<T, 1>(r[2 * j], a);
    widen<T, 1>(r[2 * j + 1], b);
    return f2(a[0], b[0]);
  }
}
template <int V>
__device__ __forceinline__ F2 rate_pair(const float (&rate)[V]) {
  return f2(rate[0], rate[V - 1]);
}

// a and sqrt(1 - a^2) sig(i) x for a pair: any channels.
__device__ __forceinline__ void any_gate(float rate0, float rate1, F2 r, F2 i, F2 x, F2& a, F2& b) {
  const Gate g0 = gate_any(lo(r), rate0), g1 = gate_any(hi(r), rate1);
  a = f2(g0.a, g1.a);
  b = f2(g0.s * sigmoid(lo(i)) * lo(x), g1.s * sigmoid(hi(i)) * hi(x));
}
// The maps of a segment's steps, P[s] h + H[s] the state after step s, as pairs
// in the order of pair_of.
template <int V, int S>
struct Steps {
  F2 P[S * V / 2], H[S * V / 2];
  __device__ __forceinline__ static float part(const F2 (&a)[S * V / 2], int k, int v) {
    const int e = k * V + v;
    return e & 1 ? hi(a[e / 2]) : lo(a[e / 2]);
  }
  __device__ __forceinline__ float p(int k, int v) const { return part(P, k, v); }
  __device__ __forceinline__ float h(int k, int v) const { return part(H, k, v); }
  // the pair j from its steps' a and b
  __device__ __forceinline__ void step(int j, F2 a, F2 b) {
    const int before = j > 0 ? j - 1 : 0;
    if constexpr (V == 2) {
      P[j] = j == 0 ? a : mul2(a, P[before]);
      H[j] = j == 0 ? b : fma2(a, H[before], b);
    } else {
      const float p0 = j == 0 ? lo(a) : lo(a) * hi(P[before]), h0 = j == 0 ? lo(b) : fmaf(lo(a), hi(H[before]), lo(b));
      P[j] = f2(p0, hi(a) * p0);
      H[j] = f2(h0, fmaf(hi(a), h0, hi(b)));
    }
  }
};
// Any channels.
template <typename T, int V, int S>
__device__ __forceinline__ void segment_maps(const Raw<T, V> (&rx)[S], const Raw<T, V> (&rr)[S], const Raw<T, V> (&ri)[S],
                                             const float (&rate)[V], Steps<V, S>& m) {
#pragma unroll
  for (int j = 0; j < S * V / 2; ++j) {
    F2 a, b;
    any_gate(rate[0], rate[V - 1], pair_of<T, V, S>(rr, j), pair_of<T, V, S>(ri, j), pair_of<T, V, S>(rx, j), a, b);
    m.step(j, a, b);
  }
}
// max(v, -60) of raw values, NaN kept: the input gate's floor; sig(-60) is 9e-27.
__device__ __forceinline__ Raw<float, 1> floor_gate(const Raw<float, 1>& r) {
  float o;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(__uint_as_float(r.w[0])), "f"(-60.f));
  return Raw<float, 1>{{__float_as_uint(o)}};
}
template <int V>
__device__ __forceinline__ Raw<__half, V> floor_gate(const Raw<__half, V>& r) {
  const __half2 o = __hmax2_nan(*reinterpret_cast<const __half2*>(&r.w[0]), __float2half2_rn(-60.f));
  return Raw<__half, V>{{*reinterpret_cast<const uint32_t*>(&o)}};
}
template <int V>
__device__ __forceinline__ Raw<__nv_bfloat16, V> floor_gate(const Raw<__nv_bfloat16, V>& r) {
  const __nv_bfloat162 o = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&r.w[0]), __float2bfloat162_rn(-60.f));
  return Raw<__nv_bfloat16, V>{{*reinterpret_cast<const uint32_t*>(&o)}};
}
// a and b = sqrt(1 - a^2) sig(i) x for a pair of slow or plain channels.
// sqrt(1 - a^2) sig(i) is taken as z / sqrt(z (1 + exp(-i))^2) with z = 1 - a^2,
// which saves a reciprocal; the constant added under the root keeps it 0 where
// z is, and the floor on i (floor_gate) keeps 0 times infinity out.  A factor
// below 1e-18 (r below -80 or i below -40) may come out as less.
template <RateKind K>
__device__ __forceinline__ void gate_pair(const GateConsts& c, F2 rates, F2 r, F2 i, F2 x, F2& a, F2& b) {
  F2 e;
  decay_pair<K>(c, mul2(rates, rcp2(one_plus_exp_neg2(c, r))), e, a);
  const F2 z = mul2(e, add2(a, c.one)), q = one_plus_exp_neg2(c, i);
  b = mul2(mul2(z, rsqrt2(fma2(mul2(z, q), q, c.tiny))), x);
}
template <RateKind K, typename T, int V, int S>
__device__ __forceinline__ void segment_maps_of(const Raw<T, V> (&rx)[S], const Raw<T, V> (&rr)[S], Raw<T, V> (&ri)[S],
                                                  F2 rates, const GateConsts& c, Steps<V, S>& m) {
#pragma unroll
  for (int k = 0; k < S; ++k) ri[k] = floor_gate(ri[k]);
#pragma unroll
  for (int j = 0; j < S * V / 2; ++j) {
    F2 a, b;
    gate_pair<K>(c, rates, pair_of<T, V, S>(rr, j), pair_of<T, V, S>(ri, j), pair_of<T, V, S>(rx, j), a, b);
    m.step(j, a, b);
  }
}
template <typename T, int V, int S>
__device__ __forceinline__ void segment_maps_by(RateKind kind, const Raw<T, V> (&rx)[S], const Raw<T, V> (&rr)[S],
                                                Raw<T, V> (&ri)[S], const float (&rate)[V], const GateConsts& c,
                                                Steps<V, S>& m) {
  if (kind == kRateSlow)
    segment_maps_of<kRateSlow, T, V, S>(rx, rr, ri, rate_pair(rate), c, m);
  else if (kind == kRatePlain || (kind == kRateSteep && all_fast<T, V, S>(rr, ri)))
    segment_maps_of<kRatePlain, T, V, S>(rx, rr, ri, rate_pair(rate), c, m);
  else
    segment_maps<T, V, S>(rx, rr, ri, rate, m);
}
// Rows `live` and on of a segment lie past the sequence's end: a gate of minus
// infinity and a zero make their steps the identity.
template <typename T, int V, int S>
__device__ __forceinline__ void mask_rows(Raw<T, V> (&rx)[S], Raw<T, V> (&rr)[S], Raw<T, V> (&ri)[S], int live) {
  constexpr uint32_t ninf = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
#pragma unroll
  for (int k = 0; k < S; ++k)
    if (k >= live) rx[k].w[0] = 0, ri[k].w[0] = 0, rr[k].w[0] = ninf;
}
// saved states and outputs of a segment from the state before it
template <typename T, int V, int S>
__device__ __forceinline__ void finish_segment(const ScanArgs& s, const Steps<V, S>& m, const float (&start)[V], int64_t t,
                                               int64_t n, T* y, float* saved) {
  if (saved != nullptr) {
#pragma unroll
    for (int k = 0; k < S; k += kChunk)
      if (t + k < n) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          saved[(int64_t)(k / kChunk) * s.D + v] =
              k == 0 ? start[v] : fmaf(m.p(k > 0 ? k - 1 : 0, v), start[v], m.h(k > 0 ? k - 1 : 0, v));
      }
  }
  const F2 from = f2(start[0], start[V - 1]);
  const int64_t step = s.sy.t;
  const bool whole = t + S <= n;
#pragma unroll
  for (int j = 0; j < S * V / 2; ++j) {
    const F2 o = fma2(m.P[j], from, m.H[j]);
    if constexpr (V == 2) {
      const float f[2] = {lo(o), hi(o)}, none[2] = {0.f, 0.f};
      if (whole || t + j < n) st_raw<T, V>(y, narrow<T, V>(f));
      else if (t + j < s.T) st_raw<T, V>(y, narrow<T, V>(none));
      y += step;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f[1] = {h ? hi(o) : lo(o)}, none[1] = {0.f};
        if (whole || t + 2 * j + h < n) st_raw<T, V>(y, narrow<T, V>(f));
        else if (t + 2 * j + h < s.T) st_raw<T, V>(y, narrow<T, V>(none));
        y += step;
      }
    }
  }
}

// The same walk with the tiles brought by TMA: boxes of W S tokens x 128 bytes
// of channels of each input in a ring of ST stages, so that loads cost the
// warps no instructions and no registers.  Thread 0 asks for a tile as soon as
// the block has passed the barrier that ends the reading of its stage.
struct ScanMaps {
  CUtensorMap x, r, i, dy;
};
template <int V, int S, int W, int ST, int NT>
struct ScanRing {
  static constexpr int kTensorBytes = W * S * 128;
  static constexpr int kStageBytes = NT * kTensorBytes;
  static constexpr int kMapsOff = ST * kStageBytes;
  static constexpr int kBarOff = kMapsOff + (int)sizeof(MapBuffers<V, W>);
  static constexpr int kBytes = kBarOff + ST * 8 + 128;  // 128: room to align the ring
};
__device__ __forceinline__ unsigned char* align128(unsigned char* p) {
  return p + ((128u - (smem_u32(p) & 127u)) & 127u);
}
// After a wait that ran out: no copy of this block is in flight when it ends.
template <int ST>
__device__ __forceinline__ void drain_ring(uint64_t* full, int rounds, const Place& at, uint64_t limit) {
  if (at.limit != 0 || threadIdx.x != 0) return;
  for (int k = rounds > ST ? rounds - ST : 0; k < rounds; ++k) mbar_wait(&full[k % ST], (uint32_t)(k / ST) & 1u, limit);
}
// S rows of a segment from its place in a stage.
template <typename T, int V, int S>
__device__ __forceinline__ void lds_rows(Raw<T, V> (&out)[S], const unsigned char* tensor, int warp, int lane) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(tensor + warp * S * 128) + lane;
#pragma unroll
  for (int k = 0; k < S; ++k) out[k].w[0] = p[k * 32];
}

template <typename T, int S, int W, int ST, int MB, bool CL>
__global__ void __launch_bounds__(32 * W, MB)
scan_fwd_tma_kernel(const __grid_constant__ ScanMaps tm, ScanArgs s, int ns, int slabs, int* status, uint64_t limit) {
  constexpr int V = 4 / sizeof(T);
  using Ring = ScanRing<V, S, W, ST, 3>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = align128(smem_raw);
  MapBuffers<V, W>& maps = *reinterpret_cast<MapBuffers<V, W>*>(ring + Ring::kMapsOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + Ring::kBarOff);
  if (threadIdx.x == 0) {
    for (int k = 0; k < ST; ++k) mbar_init(&full[k], 1);
    init_maps(maps, ns);
  }
  if constexpr (CL) cluster_arrive();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = CL ? blockIdx.x / (uint32_t)ns : blockIdx.x;
  const int rank = CL ? (int)(blockIdx.x - unit * (uint32_t)ns) : 0;
  const uint32_t b = unit / (uint32_t)slabs;
  const int d0 = (int)(unit - b * (uint32_t)slabs) * 32 * V, d = d0 + lane * V;
  const bool mine = d < s.D;
  Place at{warp, lane, rank, ns, status, limit};
  const int64_t chunks = (s.T + kChunk - 1) / kChunk;
  grid_dependency_wait();
  const int n = (int)seq_len(s.lens, b, s.T);  // the launcher keeps T below 2^30
  const int tile = ns * W * S, rounds = (int)((uint32_t)(n + tile - 1) / (uint32_t)tile);
  __syncthreads();  // the barriers are set up
  auto ask = [&](int round) {  // thread 0; a tile past the sequence's end is asked for too, so every round waits
    const int st = round % ST;
    unsigned char* to = ring + st * Ring::kStageBytes;
    mbar_arrive_expect_tx(&full[st], Ring::kStageBytes);
    const int t0 = round * tile + rank * W * S;
    tma_load_3d(to, &tm.r, &full[st], d0, t0, (int)b);
    tma_load_3d(to + Ring::kTensorBytes, &tm.i, &full[st], d0, t0, (int)b);
    tma_load_3d(to + 2 * Ring::kTensorBytes, &tm.x, &full[st], d0, t0, (int)b);
  };
  if (threadIdx.x == 0)
    for (int k = 0; k < ST && k < rounds; ++k) ask(k);
  float rate[V], carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = mine ? decay_rate(s.lam[d + v], s.decay) : 0.1f;
    carry[v] = mine && s.h0 ? s.h0[(int64_t)b * s.D + d + v] : 0.f;
  }
  int t = (rank * W + warp) * S;  // this warp's segment
  T* y = static_cast<T*>(s.y) + (int64_t)b * s.sy.b + d;
  if constexpr (CL) cluster_wait();  // every block of the cluster is ready for maps
  const RateKind kind = warp_kind<V>(rate);
  const GateConsts consts = gate_consts();
  for (int round = 0; round < rounds; ++round, t += tile) {
    const int st = round % ST;
    at.wait(&full[st], (uint32_t)(round / ST) & 1u, 70);
    Steps<V, S> m;
    float start[V], p[V], q[V];
    {
      const unsigned char* rows = ring + st * Ring::kStageBytes;
      Raw<T, V> rx[S], rr[S], ri[S];
      lds_rows<T, V, S>(rr, rows, warp, lane);
      lds_rows<T, V, S>(ri, rows + Ring::kTensorBytes, warp, lane);
      lds_rows<T, V, S>(rx, rows + 2 * Ring::kTensorBytes, warp, lane);
      if (t + S > n) mask_rows<T, V, S>(rx, rr, ri, n > t ? (int)(n - t) : 0);
      segment_maps_by<T, V, S>(kind, rx, rr, ri, rate, consts, m);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = m.p(S - 1, v), q[v] = m.h(S - 1, v);
    exchange<V, W, CL, false>(maps, (uint32_t)round, at, p, q, carry, start);
    if (threadIdx.x == 0 && round + ST < rounds) ask(round + ST);
    if (mine)
      finish_segment<T, V, S>(s, m, start, t, n, y + (int64_t)t * s.sy.t,
                              s.saved ? s.saved + (b * chunks + t / kChunk) * s.D + d : nullptr);
  }
  drain_ring<ST>(full, rounds, at, limit);
  if (mine) {
    if (s.hT != nullptr && rank == 0 && warp == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) s.hT[(int64_t)b * s.D + d + v] = carry[v];
    const float none[V] = {};
    for (; t < s.T; t += tile)
      for (int k = 0; k < S && t + k < s.T; ++k) st_raw<T, V>(y + (int64_t)(t + k) * s.sy.t, narrow<T, V>(none));
  }
  leave<CL>();
}

template <typename T, int V, int S, int W, bool CL>
__global__ void __launch_bounds__(32 * W)
scan_fwd_kernel(ScanArgs s, int ns, int slabs, int* status, uint64_t limit) {
  __shared__ MapBuffers<V, W> maps;
  if constexpr (CL) {
    if (threadIdx.x == 0) init_maps(maps, ns);
    cluster_arrive();
  }
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = CL ? blockIdx.x / (uint32_t)ns : blockIdx.x;
  const int rank = CL ? (int)(blockIdx.x - unit * (uint32_t)ns) : 0;
  const int64_t b = unit / (uint32_t)slabs;
  const int d = ((int)(unit - (uint32_t)b * (uint32_t)slabs) * 32 + lane) * V;
  const bool mine = d < s.D;
  Place at{warp, lane, rank, ns, status, limit};
  const T* x = static_cast<const T*>(s.x) + b * s.sx.b + d;
  const T* r = static_cast<const T*>(s.r) + b * s.sr.b + d;
  const T* g = static_cast<const T*>(s.i) + b * s.si.b + d;
  T* y = static_cast<T*>(s.y) + b * s.sy.b + d;
  const int64_t chunks = (s.T + kChunk - 1) / kChunk;
  grid_dependency_wait();
  const int64_t n = seq_len(s.lens, b, s.T);
  float rate[V], carry[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = mine ? decay_rate(s.lam[d + v], s.decay) : 0.1f;
    carry[v] = mine && s.h0 ? s.h0[b * s.D + d + v] : 0.f;
  }
  const RateKind kind = warp_kind<V>(rate);
  const GateConsts consts = gate_consts();
  const int64_t tile = (int64_t)ns * W * S, rounds = (n + tile - 1) / tile;
  int64_t t = ((int64_t)rank * W + warp) * S;  // this warp's segment
  Raw<T, V> rx[S], rr[S], ri[S];
  ld_rows<T, V, S>(rr, r, s.sr.t, t, n, mine);
  ld_rows<T, V, S>(ri, g, s.si.t, t, n, mine);
  ld_rows<T, V, S>(rx, x, s.sx.t, t, n, mine);
  if constexpr (CL) cluster_wait();  // every block of the cluster is ready for maps
  for (int64_t round = 0; round < rounds; ++round, t += tile) {
    Steps<V, S> m;
    float start[V], p[V], q[V];
    if (t + S > n) mask_rows<T, V, S>(rx, rr, ri, n > t ? (int)(n - t) : 0);
    segment_maps_by<T, V, S>(kind, rx, rr, ri, rate, consts, m);
    ld_rows<T, V, S>(rr, r, s.sr.t, t + tile, n, mine);
    ld_rows<T, V, S>(ri, g, s.si.t, t + tile, n, mine);
    ld_rows<T, V, S>(rx, x, s.sx.t, t + tile, n, mine);
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = m.p(S - 1, v), q[v] = m.h(S - 1, v);
    exchange<V, W, CL, false>(maps, (uint32_t)round, at, p, q, carry, start);
    if (mine)
      finish_segment<T, V, S>(s, m, start, t, n, y + t * s.sy.t,
                              s.saved ? s.saved + (b * chunks + t / kChunk) * s.D + d : nullptr);
  }
  if (mine) {
    if (s.hT != nullptr && rank == 0 && warp == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) s.hT[b * s.D + d + v] = carry[v];
    const float none[V] = {};
    for (; t < s.T; t += tile)
      for (int k = 0; k < S && t + k < s.T; ++k) st_raw<T, V>(y + (t + k) * s.sy.t, narrow<T, V>(none));
  }
  leave<CL>();
}

// ---------------------------------------------------------------------------
// Backward: the same walk from the end.  Every gradient of a token is a factor
// times g_t, the gradient of h_t, and the factors come from the inputs and the
// state before the token, which the forward pass saved for every kChunk-th one
// (S is kChunk: a segment starts from its own saved state):
//   dx = c1 g,  di = c2 g,  dr = c3 g,  dl sig(r) = c4 g
//   c1 = s sig(i);  c2 = c1 x (1 - sig(i));  c4 = a (h sig(r) - a sig(i) x k)
//   c3 = -rate (1 - sig(r)) c4
// The recurrence g_t = dy_t + a_{t+1} g_{t+1} gives g_s = G_s + Q_s u for the
// gradient u that comes into a segment from behind, so only c1 ... c3, G and Q
// are kept, and dlam's share is sum c4 G + u sum c4 Q.
// ---------------------------------------------------------------------------
template <int V, int S>
struct Factors {
  F2 c1[S * V / 2], c2[S * V / 2], c3[S * V / 2], G[S * V / 2], Q[S * V / 2];  // pairs in the order of pair_of
  float outp[V], outq[V];  // the map of a segment: u -> outp u + outq
  float sumG[V], sumQ[V];
};

// Two pairs of channels' sums, or the pair of one channel's two tokens added.
template <int V>
__device__ __forceinline__ void unpair(F2 s, float (&out)[V]) {
  if constexpr (V == 2)
    out[0] = lo(s), out[1] = hi(s);
  else
    out[0] = lo(s) + hi(s);
}

// a, the factors and c4 of a pair of steps: any channels and gates.  h: the state
// before a token; it moves on.
struct StepFactors {
  F2 a, c1, c2, c3, c4;
};
template <int V>
__device__ __forceinline__ StepFactors factors_any(const float (&rate)[V], F2 r, F2 i, F2 x, float (&h)[V]) {
  float a[2], c1[2], c2[2], c3[2], c4[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int v = V == 2 ? e : 0;
    const float xv = e ? hi(x) : lo(x);
    const Gate q = gate_any(e ? hi(r) : lo(r), rate[v]);
    float si, so;
    sigmoid_pair(e ? hi(i) : lo(i), si, so);
    a[e] = q.a;
    c1[e] = q.s * si;
    const float b = c1[e] * xv;
    c2[e] = b * so;
    c4[e] = q.a * fmaf(h[v], q.g, -(q.a * si) * (xv * q.k));
    c3[e] = -rate[v] * q.o * c4[e];
    h[v] = fmaf(q.a, h[v], b);
  }
  return {f2(a[0], a[1]), f2(c1[0], c1[1]), f2(c2[0], c2[1]), f2(c3[0], c3[1]), f2(c4[0], c4[1])};
}
// Slow or plain channels and ordinary gates (all_fast): one reciprocal for both
// logistic functions, u = 1 / (D q), sig(r) = u q, sig(i) = u D; 1 - sig is exp(-v)
// times sig, because a difference from 1 loses the gradients of open gates (from 17
// on all of them).
template <RateKind K, int V>
__device__ __forceinline__ StepFactors factors_fast(const GateConsts& c, F2 rates, F2 r, F2 i, F2 x, float (&h)[V]) {
  const F2 er = exp_neg2(c, r), ei = exp_neg2(c, i), D = add2(er, c.one), q = add2(ei, c.one), u = rcp2(mul2(D, q));
  const F2 g = mul2(u, q), si = mul2(u, D);
  StepFactors f;
  F2 e;
  decay_pair<K>(c, mul2(rates, g), e, f.a);
  const F2 z = mul2(e, add2(f.a, c.one)), inv = rsqrt2(z);
  f.c1 = mul2(mul2(z, inv), si);
  const F2 b = mul2(f.c1, x);
  f.c2 = mul2(b, mul2(ei, si));
  const F2 t = mul2(mul2(f.a, si), mul2(mul2(x, c.none), mul2(g, inv)));
  F2 before;
  if constexpr (V == 2) {
    before = f2(h[0], h[1]);
    const F2 after = fma2(f.a, before, b);
    h[0] = lo(after), h[1] = hi(after);
  } else {
    const float mid = fmaf(lo(f.a), h[0], lo(b));
    before = f2(h[0], mid);
    h[0] = fmaf(hi(f.a), mid, hi(b));
  }
  f.c4 = mul2(f.a, fma2(before, g, t));
  f.c3 = mul2(mul2(mul2(rates, c.none), mul2(er, g)), f.c4);
  return f;
}

// Rows past the sequence's end have passed mask_rows: a is 1 and every factor 0.
template <typename T, int V, int S>
__device__ __forceinline__ void segment_factors(const Raw<T, V> (&rx)[S], const Raw<T, V> (&rr)[S],
                                                const Raw<T, V> (&ri)[S], const Raw<T, V> (&rg)[S], const float (&rate)[V],
                                                const float (&h0)[V], RateKind kind, const GateConsts& c, Factors<V, S>& f) {
  constexpr int N = S * V / 2;
  F2 a[N], c4[N];
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = h0[v];
  auto fast = [&](auto k) {
    constexpr RateKind K = decltype(k)::value;
    const F2 rates = rate_pair(rate);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const StepFactors q = factors_fast<K, V>(c, rates, pair_of<T, V, S>(rr, j), pair_of<T, V, S>(ri, j), pair_of<T, V, S>(rx, j), h);
      a[j] = q.a, f.c1[j] = q.c1, f.c2[j] = q.c2, f.c3[j] = q.c3, c4[j] = q.c4;
    }
  };
  if (__builtin_expect(kind == kRateSlow, 1)) {
    fast(std::integral_constant<RateKind, kRateSlow>{});
  } else if (kind != kRateAny) {
    fast(std::integral_constant<RateKind, kRatePlain>{});
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const StepFactors q = factors_any<V>(rate, pair_of<T, V, S>(rr, j), pair_of<T, V, S>(ri, j), pair_of<T, V, S>(rx, j), h);
      a[j] = q.a, f.c1[j] = q.c1, f.c2[j] = q.c2, f.c3[j] = q.c3, c4[j] = q.c4;
    }
  }
  F2 sG = c.zero, sQ = c.zero;
#pragma unroll
  for (int j = N - 1; j >= 0; --j) {
    const F2 dy = pair_of<T, V, S>(rg, j);
    const int k = j + 1 < N ? j + 1 : j;
    if constexpr (V == 2) {
      f.G[j] = j == N - 1 ? dy : fma2(a[k], f.G[k], dy);
      f.Q[j] = j == N - 1 ? c.one : mul2(a[k], f.Q[k]);
    } else {
      const float g1 = j == N - 1 ? hi(dy) : fmaf(lo(a[k]), lo(f.G[k]), hi(dy)), q1 = j == N - 1 ? 1.f : lo(a[k]) * lo(f.Q[k]);
      f.G[j] = f2(fmaf(hi(a[j]), g1, lo(dy)), g1);
      f.Q[j] = f2(hi(a[j]) * q1, q1);
    }
    sG = fma2(c4[j], f.G[j], sG);
    sQ = fma2(c4[j], f.Q[j], sQ);
  }
  unpair<V>(sG, f.sumG);
  unpair<V>(sQ, f.sumQ);
  const F2 op = mul2(a[0], f.Q[0]), oq = mul2(a[0], f.G[0]);
#pragma unroll
  for (int v = 0; v < V; ++v) f.outp[v] = v ? hi(op) : lo(op), f.outq[v] = v ? hi(oq) : lo(oq);
}

// dx, dr, di of a segment from the gradient u behind it.
template <typename T, int V, int S>
__device__ __forceinline__ void finish_factors(const ScanArgs& s, const Factors<V, S>& f, const float (&u)[V], int64_t t,
                                               int64_t n, T* dx, T* dr, T* di) {
  const F2 from = f2(u[0], u[V - 1]);
  const bool whole = t + S <= n;
  auto put = [&](int64_t at, const Raw<T, V>& ox, const Raw<T, V>& orr, const Raw<T, V>& oi) {
    if (whole || at < n) {
      st_raw<T, V>(dx, ox), st_raw<T, V>(dr, orr), st_raw<T, V>(di, oi);
    } else if (at < s.T) {
      st_raw<T, V>(dx, zero_raw<T, V>()), st_raw<T, V>(dr, zero_raw<T, V>()), st_raw<T, V>(di, zero_raw<T, V>());
    }
    dx += s.sx.t, dr += s.sr.t, di += s.si.t;
  };
#pragma unroll
  for (int j = 0; j < S * V / 2; ++j) {
    const F2 g = fma2(f.Q[j], from, f.G[j]);
    const F2 ox = mul2(f.c1[j], g), oi = mul2(f.c2[j], g), orr = mul2(f.c3[j], g);
    if constexpr (V == 2) {
      const float a[2] = {lo(ox), hi(ox)}, b[2] = {lo(orr), hi(orr)}, c[2] = {lo(oi), hi(oi)};
      put(t + j, narrow<T, V>(a), narrow<T, V>(b), narrow<T, V>(c));
    } else {
      const float a[1] = {lo(ox)}, b[1] = {lo(orr)}, c[1] = {lo(oi)}, d[1] = {hi(ox)}, e[1] = {hi(orr)}, g1[1] = {hi(oi)};
      put(t + 2 * j, narrow<T, V>(a), narrow<T, V>(b), narrow<T, V>(c));
      put(t + 2 * j + 1, narrow<T, V>(d), narrow<T, V>(e), narrow<T, V>(g1));
    }
  }
}

// The block's partial sum of dlam, its warps in order, and dh0.
template <int V, int W>
__device__ __forceinline__ void finish_block(const ScanArgs& s, MapBuffers<V, W>& maps, const Place& at, int64_t b, int d,
                                             bool mine, const float (&dsum)[V], const float (&carry)[V]) {
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) maps.warp[0][at.warp][at.lane].p[v] = dsum[v];
  __syncthreads();
  if (at.warp == 0 && mine) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) sum += maps.warp[0][k][at.lane].p[v];
      s.ws[(b * at.ns + at.rank) * s.D + d + v] = sum;
      if (s.dh0 != nullptr && at.rank == 0) s.dh0[b * s.D + d + v] = carry[v];
    }
  }
}

template <typename T, int W, int ST, int MB, bool CL>
__global__ void __launch_bounds__(32 * W, MB)
scan_bwd_tma_kernel(const __grid_constant__ ScanMaps tm, ScanArgs s, int ns, int slabs, int* status, uint64_t limit) {
  constexpr int V = 4 / sizeof(T), S = kChunk;
  using Ring = ScanRing<V, S, W, ST, 4>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = align128(smem_raw);
  MapBuffers<V, W>& maps = *reinterpret_cast<MapBuffers<V, W>*>(ring + Ring::kMapsOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + Ring::kBarOff);
  if (threadIdx.x == 0) {
    for (int k = 0; k < ST; ++k) mbar_init(&full[k], 1);
    init_maps(maps, ns);
  }
  if constexpr (CL) cluster_arrive();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = CL ? blockIdx.x / (uint32_t)ns : blockIdx.x;
  const int rank = CL ? (int)(blockIdx.x - unit * (uint32_t)ns) : 0;
  const uint32_t b = unit / (uint32_t)slabs;
  const int d0 = (int)(unit - b * (uint32_t)slabs) * 32 * V, d = d0 + lane * V;
  const bool mine = d < s.D;
  Place at{warp, lane, rank, ns, status, limit};
  const int64_t chunks = (s.T + kChunk - 1) / kChunk;
  grid_dependency_wait();
  const int n = (int)seq_len(s.lens, b, s.T);  // the launcher keeps T below 2^30
  const int tile = ns * W * S, rounds = (int)((uint32_t)(n + tile - 1) / (uint32_t)tile);
  const int first = (rank * W + warp) * S;
  __syncthreads();  // the barriers are set up
  auto ask = [&](int round) {  // thread 0
    const int st = round % ST;
    unsigned char* to = ring + st * Ring::kStageBytes;
    mbar_arrive_expect_tx(&full[st], Ring::kStageBytes);
    const int t0 = (rounds - 1 - round) * tile + rank * W * S;
    tma_load_3d(to, &tm.r, &full[st], d0, t0, (int)b);
    tma_load_3d(to + Ring::kTensorBytes, &tm.i, &full[st], d0, t0, (int)b);
    tma_load_3d(to + 2 * Ring::kTensorBytes, &tm.x, &full[st], d0, t0, (int)b);
    tma_load_3d(to + 3 * Ring::kTensorBytes, &tm.dy, &full[st], d0, t0, (int)b);
  };
  if (threadIdx.x == 0)
    for (int k = 0; k < ST && k < rounds; ++k) ask(k);
  T* dx = static_cast<T*>(s.dx) + (int64_t)b * s.sx.b + d;
  T* dr = static_cast<T*>(s.dr) + (int64_t)b * s.sr.b + d;
  T* di = static_cast<T*>(s.di) + (int64_t)b * s.si.b + d;
  float rate[V], carry[V], dsum[V], h0[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = mine ? decay_rate(s.lam[d + v], s.decay) : 0.1f;
    carry[v] = mine && s.dhT ? s.dhT[(int64_t)b * s.D + d + v] : 0.f;
    dsum[v] = 0.f;
  }
  if (mine) {  // past the end: zeros
    const float none[V] = {};
    for (int t = rounds * tile + first; t < s.T; t += tile)
      for (int k = 0; k < S && t + k < s.T; ++k) {
        st_raw<T, V>(dx + (int64_t)(t + k) * s.sx.t, narrow<T, V>(none));
        st_raw<T, V>(dr + (int64_t)(t + k) * s.sr.t, narrow<T, V>(none));
        st_raw<T, V>(di + (int64_t)(t + k) * s.si.t, narrow<T, V>(none));
      }
  }
  const float* saved = s.saved + b * chunks * s.D + d;
  int t = (rounds - 1) * tile + first;
  auto state_at = [&](int at_t) {
#pragma unroll
    for (int v = 0; v < V; ++v) h0[v] = mine && at_t >= 0 && at_t < n ? saved[(int64_t)(at_t / kChunk) * s.D + v] : 0.f;
  };
  state_at(t);
  const RateKind kind = warp_kind<V>(rate);
  const GateConsts consts = gate_consts();
  if constexpr (CL) cluster_wait();  // every block of the cluster is ready for maps
  for (int round = 0; round < rounds; ++round, t -= tile) {
    const int st = round % ST;
    at.wait(&full[st], (uint32_t)(round / ST) & 1u, 73);
    Factors<V, S> f;
    float u[V];
    {
      const unsigned char* rows = ring + st * Ring::kStageBytes;
      Raw<T, V> rx[S], rr[S], ri[S], rg[S];
      lds_rows<T, V, S>(rr, rows, warp, lane);
      lds_rows<T, V, S>(ri, rows + Ring::kTensorBytes, warp, lane);
      lds_rows<T, V, S>(rx, rows + 2 * Ring::kTensorBytes, warp, lane);
      lds_rows<T, V, S>(rg, rows + 3 * Ring::kTensorBytes, warp, lane);
      if (t + S > n) {
        const int live = n > t ? n - t : 0;
        mask_rows<T, V, S>(rx, rr, ri, live);
#pragma unroll
        for (int k = 0; k < S; ++k)
          if (k >= live) rg[k].w[0] = 0;
      }
      segment_factors<T, V, S>(rx, rr, ri, rg, rate, h0, all_fast<T, V, S>(rr, ri) ? kind : kRateAny, consts, f);
    }
    state_at(t - tile);
    exchange<V, W, CL, true>(maps, (uint32_t)round, at, f.outp, f.outq, carry, u);
    if (threadIdx.x == 0 && round + ST < rounds) ask(round + ST);
    if (mine)
      finish_factors<T, V, S>(s, f, u, t, n, dx + (int64_t)t * s.sx.t, dr + (int64_t)t * s.sr.t, di + (int64_t)t * s.si.t);
#pragma unroll
    for (int v = 0; v < V; ++v) dsum[v] += fmaf(f.sumQ[v], u[v], f.sumG[v]);
  }
  drain_ring<ST>(full, rounds, at, limit);
  finish_block<V, W>(s, maps, at, b, d, mine, dsum, carry);
  leave<CL>();
}

// The same without TMA, for any alignment: rows by loads a round ahead.
template <typename T, int V, int W, bool CL>
__global__ void __launch_bounds__(32 * W)
scan_bwd_kernel(ScanArgs s, int ns, int slabs, int* status, uint64_t limit) {
  constexpr int S = kChunk;
  __shared__ MapBuffers<V, W> maps;
  if constexpr (CL) {
    if (threadIdx.x == 0) init_maps(maps, ns);
    cluster_arrive();
  }
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = CL ? blockIdx.x / (uint32_t)ns : blockIdx.x;
  const int rank = CL ? (int)(blockIdx.x - unit * (uint32_t)ns) : 0;
  const int64_t b = unit / (uint32_t)slabs;
  const int d = ((int)(unit - (uint32_t)b * (uint32_t)slabs) * 32 + lane) * V;
  const bool mine = d < s.D;
  Place at{warp, lane, rank, ns, status, limit};
  const T* x = static_cast<const T*>(s.x) + b * s.sx.b + d;
  const T* r = static_cast<const T*>(s.r) + b * s.sr.b + d;
  const T* g = static_cast<const T*>(s.i) + b * s.si.b + d;
  const T* dy = static_cast<const T*>(s.dy) + b * s.sy.b + d;
  T* dx = static_cast<T*>(s.dx) + b * s.sx.b + d;
  T* dr = static_cast<T*>(s.dr) + b * s.sr.b + d;
  T* di = static_cast<T*>(s.di) + b * s.si.b + d;
  const int64_t chunks = (s.T + kChunk - 1) / kChunk;
  const float* saved = s.saved + b * chunks * s.D + d;
  grid_dependency_wait();
  const int64_t n = seq_len(s.lens, b, s.T);
  float rate[V], carry[V], dsum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = mine ? decay_rate(s.lam[d + v], s.decay) : 0.1f;
    carry[v] = mine && s.dhT ? s.dhT[b * s.D + d + v] : 0.f;
    dsum[v] = 0.f;
  }
  const RateKind kind = warp_kind<V>(rate);
  const GateConsts consts = gate_consts();
  const int64_t tile = (int64_t)ns * W * S, rounds = (n + tile - 1) / tile;
  const int64_t first = ((int64_t)rank * W + warp) * S;
  if (mine) {  // past the end: zeros
    const float none[V] = {};
    for (int64_t t = rounds * tile + first; t < s.T; t += tile)
      for (int k = 0; k < S && t + k < s.T; ++k) {
        st_raw<T, V>(dx + (t + k) * s.sx.t, narrow<T, V>(none));
        st_raw<T, V>(dr + (t + k) * s.sr.t, narrow<T, V>(none));
        st_raw<T, V>(di + (t + k) * s.si.t, narrow<T, V>(none));
      }
  }
  int64_t t = (rounds - 1) * tile + first;
  Raw<T, V> rx[S], rr[S], ri[S], rg[S];
  float h0[V];
  auto load = [&](int64_t at) {
    const int64_t end = at >= 0 ? n : 0;  // the walk's last prefetch lies before the sequence
    at = at >= 0 ? at : 0;
    ld_rows<T, V, S>(rr, r, s.sr.t, at, end, mine);
    ld_rows<T, V, S>(ri, g, s.si.t, at, end, mine);
    ld_rows<T, V, S>(rx, x, s.sx.t, at, end, mine);
    ld_rows<T, V, S>(rg, dy, s.sy.t, at, end, mine);
#pragma unroll
    for (int v = 0; v < V; ++v) h0[v] = mine && at < end ? saved[at / kChunk * s.D + v] : 0.f;
  };
  load(t);
  if constexpr (CL) cluster_wait();  // every block of the cluster is ready for maps
  for (int64_t round = 0; round < rounds; ++round, t -= tile) {
    Factors<V, S> f;
    float u[V];
    if (t + S > n) {
      const int live = n > t ? (int)(n - t) : 0;
      mask_rows<T, V, S>(rx, rr, ri, live);
#pragma unroll
      for (int k = 0; k < S; ++k)
        if (k >= live) rg[k].w[0] = 0;
    }
    segment_factors<T, V, S>(rx, rr, ri, rg, rate, h0, all_fast<T, V, S>(rr, ri) ? kind : kRateAny, consts, f);
    load(t - tile);
    exchange<V, W, CL, true>(maps, (uint32_t)round, at, f.outp, f.outq, carry, u);
    if (mine) finish_factors<T, V, S>(s, f, u, t, n, dx + t * s.sx.t, dr + t * s.sr.t, di + t * s.si.t);
#pragma unroll
    for (int v = 0; v < V; ++v) dsum[v] += fmaf(f.sumQ[v], u[v], f.sumG[v]);
  }
  finish_block<V, W>(s, maps, at, b, d, mine, dsum, carry);
  leave<CL>();
}

// dlam[d] = -c sig(lam[d]) * sum of the partial rows.
__global__ void __launch_bounds__(32 * kSumRows)
scan_dlam_kernel(const float* ws, int64_t parts, int D, const float* lam, float c, float* dlam) {
  allow_dependent_launch();
  const int64_t col = blockIdx.x * 32ll + threadIdx.x;
  grid_dependency_wait();
  const float sum = column_sum(ws, parts, D, col);
  if (threadIdx.y == 0 && col < D) dlam[col] = -c * sum / (1.f + expf(-lam[col]));
}

// Launch with a cluster of ns blocks along x (1: none).
template <typename K, typename... Args>
cudaError_t launch_scan(K kernel, int64_t blocks, int threads, size_t smem, int ns, const LaunchArgs& a, Args&&... args) {
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (ns > 8) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ns, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ns > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Blocks that share a slab: as many as keep the whole grid resident at `blocks` an
// SM, while the sequence still fills a round.  Measured over 1 ... 12 (us):
//   forward, 3 an SM: 1 x 32768 x 2048 12: 131, 8: 180, 4: 277, 1: 717;
//     1 x 16384 x 2048 12: 70, 8: 92; 3 x 1537 x 700 fp32 6: 15, 8: 22, 1: 30;
//     32 x 256 x 1024 1: 20, 2: 24
//   backward, 1 an SM (2 for fp32, which holds half the channels): 1 x 16384 x 2048 4: 131, 8: 203, 1: 541;
//     2 x 4096 x 1024 4: 38, 8: 60, 1: 145; 8 x 2048 x 2048 1: 104, 2: 140; 3 x 1537 x 700 fp32 4: 27, 1: 50
int split_of(int64_t units, int64_t T, int tokens, int sms, int blocks) {
  int ns = 1;
  while (ns < kMaxSplit && units * (ns + 1) <= (int64_t)blocks * sms && (int64_t)ns * tokens < T) ++ns;
  return ns;
}

// The forward pass's split.  Two blocks a slab also pay where they overflow the GPU by
// up to a sixth, for 16-bit types and sequences of a dozen rounds and more.  One
// block / two, us, on 152 SMs, at 232, 256, 264 and 304 units (slabs of all sequences):
//   16 bits, 512 tokens   21.5 / 21.8  21.8 / 23.8    21.8 / 24.6    22.0 / 25.4
//   768                   30.3 / 28.9  30.7 / 29.9
//   2048                  74.4 / 67.6  74.9 / 68.6    75.0 / 69.3    73.6 / 74.7
//   8192                  285 / 251    287 / 253      287 / 253      226 / 257
//   fp32, 2048            49.5 / 57.9  49.8 / 62.2    50.2 / 62.6    52.3 / 65.2
template <typename T>
int fwd_split(int64_t units, int64_t tokens_all, int tokens, int sms) {
  const int ns = split_of(units, tokens_all, tokens, sms, 3);
  return ns == 1 && sizeof(T) == 2 && 4 * units <= 7 * (int64_t)sms && tokens_all >= 12 * tokens ? 2 : ns;
}

bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Tensor map of a [B, T, D] tensor for boxes of `tokens` x 128 bytes; false
// where TMA cannot take it (16-byte addresses and strides, extents of 31 bits).
template <typename T>
bool tensor_map(CUtensorMap* map, const void* p, const ScanArgs& s, SeqStride st, int tokens) {
  constexpr int es = sizeof(T);
  if (!aligned(p, 16) || st.b * es % 16 != 0 || st.t * es % 16 != 0) return false;
  if (st.b * es >= (int64_t)1 << 40 || st.t * es >= (int64_t)1 << 40) return false;
  const uint64_t dims[3] = {(uint64_t)s.D, (uint64_t)s.T, (uint64_t)s.B};
  const uint64_t strides[2] = {(uint64_t)(st.t * es), (uint64_t)(st.b * es)};
  const uint32_t box[3] = {128 / es, (uint32_t)tokens, 1}, ones[3] = {1, 1, 1};
  const CUtensorMapDataType type = es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  return encode_tiled(map, type, 3, p, dims, strides, box, ones) == CUDA_SUCCESS;
}

// Whether the TMA kernels take a call: pairs of 16-bit channels in every
// output row, tokens and their strides within 31 bits.  (The inputs are
// checked by tensor_map.)
template <typename T>
bool tma_ok(const ScanArgs& s, SeqStride o, const void* p) {
  constexpr int V = 4 / sizeof(T);
  return s.D % V == 0 && o.b % V == 0 && o.t % V == 0 && aligned(p, 4) && s.T < (int64_t)1 << 30 &&
         o.t < (int64_t)1 << 27 && s.B < (int64_t)1 << 31;
}

template <typename T, int S, int W, int ST, int MB>
cudaError_t fwd_tma(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int V = 4 / sizeof(T), tokens = W * S;
  using Ring = ScanRing<V, S, W, ST, 3>;
  ScanMaps tm;
  if (!tma_ok<T>(s, s.sy, s.y) || !tensor_map<T>(&tm.x, s.x, s, s.sx, tokens) ||
      !tensor_map<T>(&tm.r, s.r, s, s.sr, tokens) || !tensor_map<T>(&tm.i, s.i, s, s.si, tokens))
    return cudaErrorNotSupported;
  const int slabs = (s.D + 32 * V - 1) / (32 * V);
  const int64_t units = s.B * slabs;
  const int ns = fwd_split<T>(units, s.T, tokens, dev.num_sms);
  if (ns == 1)
    return launch_scan(scan_fwd_tma_kernel<T, S, W, ST, MB, false>, units, 32 * W, Ring::kBytes, 1, a, tm, s, ns, slabs,
                       a.status, a.wait_limit_ns);
  return launch_scan(scan_fwd_tma_kernel<T, S, W, ST, MB, true>, units * ns, 32 * W, Ring::kBytes, ns, a, tm, s, ns, slabs,
                     a.status, a.wait_limit_ns);
}

template <typename T, int V>
cudaError_t fwd_v(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int S = 8, W = 8;
  const int slabs = (s.D + 32 * V - 1) / (32 * V);
  const int64_t units = s.B * slabs;
  const int ns = split_of(units, s.T, S * W, dev.num_sms, 3);
  if (ns == 1) return launch_scan(scan_fwd_kernel<T, V, S, W, false>, units, 32 * W, 0, 1, a, s, ns, slabs, a.status, a.wait_limit_ns);
  return launch_scan(scan_fwd_kernel<T, V, S, W, true>, units * ns, 32 * W, 0, ns, a, s, ns, slabs, a.status, a.wait_limit_ns);
}

cudaError_t sum_dlam(const ScanArgs& s, const LaunchArgs& a, int ns) {
  return launch_kernel(scan_dlam_kernel, dim3((unsigned)((s.D + 31) / 32)), dim3(32, kSumRows), 0, a,
                       (const float*)s.ws, s.B * ns, s.D, s.lam, s.decay, s.dlam);
}

template <typename T, int W, int ST, int MB, bool CL>
cudaError_t bwd_tma(const ScanArgs& s, const LaunchArgs& a, int ns) {
  constexpr int V = 4 / sizeof(T), tokens = W * kChunk;
  using Ring = ScanRing<V, kChunk, W, ST, 4>;
  ScanMaps tm;
  if (!tma_ok<T>(s, s.sx, s.dx) || !tma_ok<T>(s, s.sr, s.dr) || !tma_ok<T>(s, s.si, s.di) ||
      !tensor_map<T>(&tm.x, s.x, s, s.sx, tokens) || !tensor_map<T>(&tm.r, s.r, s, s.sr, tokens) ||
      !tensor_map<T>(&tm.i, s.i, s, s.si, tokens) || !tensor_map<T>(&tm.dy, s.dy, s, s.sy, tokens))
    return cudaErrorNotSupported;
  const int slabs = (s.D + 32 * V - 1) / (32 * V);
  const cudaError_t e = launch_scan(scan_bwd_tma_kernel<T, W, ST, MB, CL>, s.B * slabs * ns, 32 * W, Ring::kBytes, ns, a, tm,
                                    s, ns, slabs, a.status, a.wait_limit_ns);
  return e != cudaSuccess ? e : sum_dlam(s, a, ns);
}
// Eight warps, one block an SM, or (slabs enough without a cluster) six warps
// and two blocks: 8 x 2048 x 2048 104 us against 116, 4 x 8192 x 2560 371 against
// 433, 8 x 2048 x 1024 fp32 82 against 91.  Short sequences keep the larger tile:
// 32 x 256 x 1024 40 against 48, 16 x 512 x 512 fp32 24 against 28.
template <typename T>
cudaError_t bwd_by(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int V = 4 / sizeof(T), W = 8;
  const int64_t units = s.B * ((s.D + 32 * V - 1) / (32 * V));
  const int ns = split_of(units, s.T, W * kChunk, dev.num_sms, sizeof(T) == 4 ? 2 : 1);
  if (ns > 1) return bwd_tma<T, W, 3, 1, true>(s, a, ns);
  return s.T >= 1024 ? bwd_tma<T, 6, 2, 2, false>(s, a, 1) : bwd_tma<T, W, 3, 1, false>(s, a, 1);
}

template <typename T, int V>
cudaError_t bwd_v(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int W = 8;
  const int slabs = (s.D + 32 * V - 1) / (32 * V);
  const int64_t units = s.B * slabs;
  const int ns = split_of(units, s.T, kChunk * W, dev.num_sms, 1);
  const cudaError_t e = ns == 1 ? launch_scan(scan_bwd_kernel<T, V, W, false>, units, 32 * W, 0, 1, a, s, ns, slabs,
                                              a.status, a.wait_limit_ns)
                                : launch_scan(scan_bwd_kernel<T, V, W, true>, units * ns, 32 * W, 0, ns, a, s, ns, slabs,
                                              a.status, a.wait_limit_ns);
  return e != cudaSuccess ? e : sum_dlam(s, a, ns);
}

template <typename T>
cudaError_t fwd(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  if (s.T == 1) {
    const int block = 128;
    return launch_kernel(scan_step_kernel<T>, dim3((unsigned)((s.B * s.D + block - 1) / block)), dim3(block), 0, a, s);
  }
  const cudaError_t e = fwd_tma<T, 16, 4, 2, 1>(s, a, dev);
  return e == cudaErrorNotSupported ? fwd_v<T, 1>(s, a, dev) : e;
}

template <typename T>
cudaError_t bwd(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  const cudaError_t e = bwd_by<T>(s, a, dev);
  return e == cudaErrorNotSupported ? bwd_v<T, 1>(s, a, dev) : e;
}

}  // namespace

int64_t scan_saved_bytes(int64_t B, int64_t T, int D) { return B * ((T + kChunk - 1) / kChunk) * D * 4; }
// one partial row of dlam for each block that shares a slab
int64_t scan_bwd_workspace_bytes(int64_t B, int64_t T, int D) { return B * kMaxSplit * D * 4; }

cudaError_t scan_fwd_launch(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (a.dt) {
    case kF32: return fwd<float>(s, a, dev);
    case kF16: return fwd<__half>(s, a, dev);
    default: return fwd<__nv_bfloat16>(s, a, dev);
  }
}

cudaError_t scan_bwd_launch(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (a.dt) {
    case kF32: return bwd<float>(s, a, dev);
    case kF16: return bwd<__half>(s, a, dev);
    default: return bwd<__nv_bfloat16>(s, a, dev);
  }
}

}  // namespace gconv
