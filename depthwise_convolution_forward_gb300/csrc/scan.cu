// Gated linear recurrence (gconv_gated_scan_fwd / _bwd).
//
//   l_t = -c softplus(lam) sig(r_t),  a_t = exp(l_t)
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sig(i_t) x_t
//
// Each channel of each sequence is its own recurrence.
#include <initializer_list>

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

// rate = c * softplus(lam): once for each channel.
__device__ __forceinline__ float decay_rate(float lam, float c) {
  return c * (lam > 0.f ? lam + log1pf(expf(-lam)) : log1pf(expf(lam)));
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

// What the decay gate's value v gives: g = sig(v), a = exp(-rate g),
// s = sqrt(1 - a^2) and k = g / s (0 where s is 0), the factor that the
// gradient of s needs.  1 - a^2 = -e (2 + e) with e = a - 1.
struct Gate {
  float g, a, s, k;
};
// Slow channels and ordinary gates (fast_rate(rate) and v >= kFastGate): |l| is
// at most kSmall, and nothing comes near the smallest normal number.
constexpr float kFastGate = -60.f;
__device__ __forceinline__ bool fast_rate(float rate) { return rate <= kSmall && rate >= 1e-9f; }
__device__ __forceinline__ Gate gate_fast(float v, float rate) {
  Gate q;
  q.g = sigmoid(v);
  const float e = expm1_small(-rate * q.g);
  q.a = 1.f + e;
  const float z = fmaf(-e, e, -2.f * e), inv = rsqrt_approx(z);
  q.s = z * inv;
  q.k = q.g * inv;
  return q;
}
// Any channel and gate.  Far from 0, a comes from exp itself (1 + e would lose
// a small a).  For a gate below exp(-40), s and k come from sig(v) = exp(v)
// and 1 - a^2 = 2 rate sig(v), by exp(v / 2), because sig(v) and l
// themselves may be subnormal.
__device__ __forceinline__ Gate gate_any(float v, float rate) {
  Gate q;
  const float t = __expf(-fabsf(v)), w = __fdividef(1.f, 1.f + t);
  q.g = v >= 0.f ? w : t * w;
  const float l = -rate * q.g;
  const bool near = l > -kSmall;
  const float e0 = expm1_small(l), a0 = __expf(l);
  const float e = near ? e0 : a0 - 1.f;
  q.a = near ? 1.f + e0 : a0;
  const float z = fmaf(-e, e, -2.f * e);
  q.s = sqrtf(z);
  q.k = z > 0.f ? q.g / q.s : 0.f;
  if (v < -40.f && rate < 1e6f) {
    const float half = expf(0.5f * v), root = sqrtf(2.f * rate);
    q.s = half * root;
    q.k = root > 0.f ? half / root : 0.f;
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
// travel through distributed shared memory, one cluster barrier a round (two
// buffers: a block can be a round ahead of another, not two).
// ---------------------------------------------------------------------------
constexpr int kMaxSplit = 8;  // largest portable cluster

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores v at the place of `p` in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ void st_cluster(float* p, int rank, float v) {
  uint32_t to;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
}

// Maps h -> p h + q of the segments of a block and of the blocks of a cluster.
template <int V, int W>
struct MapBuffers {
  float warp[2][W][2 * V][32];
  float block[2][kMaxSplit][2 * V][32];
};

// The maps of a round: publishes this warp's (p, q), and gives the carried
// value before its segment.  `carry` moves on to the value after the round.
// REV: the order is from the last block and warp to the first.
template <int V, int W, bool CL, bool REV>
__device__ __forceinline__ void exchange(MapBuffers<V, W>& m, int buf, int warp, int lane, int rank, int ns,
                                         const float (&p)[V], const float (&q)[V], float (&carry)[V], float (&start)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) m.warp[buf][warp][2 * v][lane] = p[v], m.warp[buf][warp][2 * v + 1][lane] = q[v];
  __syncthreads();
  if constexpr (!CL) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int o = REV ? W - 1 - k : k;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (o == warp) start[v] = carry[v];
        carry[v] = fmaf(m.warp[buf][o][2 * v][lane], carry[v], m.warp[buf][o][2 * v + 1][lane]);
      }
    }
  } else {
    float bp[V], bq[V], sp[V], sq[V];  // the block's map, and the one before this warp
#pragma unroll
    for (int v = 0; v < V; ++v) bp[v] = 1.f, bq[v] = 0.f, sp[v] = 1.f, sq[v] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int o = REV ? W - 1 - k : k;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (o == warp) sp[v] = bp[v], sq[v] = bq[v];
        const float wp = m.warp[buf][o][2 * v][lane];
        bq[v] = fmaf(wp, bq[v], m.warp[buf][o][2 * v + 1][lane]);
        bp[v] *= wp;
      }
    }
    // warp w tells block w (and w + W, ...) of the cluster
    for (int to = warp; to < ns; to += W)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        st_cluster(&m.block[buf][rank][2 * v][lane], to, bp[v]);
        st_cluster(&m.block[buf][rank][2 * v + 1][lane], to, bq[v]);
      }
    cluster_arrive();
    cluster_wait();
    float base[V];
#pragma unroll
    for (int v = 0; v < V; ++v) base[v] = carry[v];
    for (int k = 0; k < ns; ++k) {
      const int o = REV ? ns - 1 - k : k;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (o == rank) base[v] = carry[v];
        carry[v] = fmaf(m.block[buf][o][2 * v][lane], carry[v], m.block[buf][o][2 * v + 1][lane]);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) start[v] = fmaf(sp[v], base[v], sq[v]);
  }
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

// Whether all gates of a warp's segment, and its channels, are ordinary ones.
template <typename T, int V, int S>
__device__ __forceinline__ bool all_fast(const Raw<T, V> (&r)[S], bool rates) {
  typename Low<T>::type m = Low<T>::zero();
#pragma unroll
  for (int k = 0; k < S; ++k) m = lowest(m, r[k]);
  return __all_sync(0xffffffffu, rates && Low<T>::get(m) >= kFastGate);
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

// The maps of a segment's steps: P[s] h + H[s] is the state after step s.
// sqrt(1 - a^2) sig(i) of an ordinary gate is z / sqrt(z (1 + exp(-i))^2),
// which saves a reciprocal.
template <bool FAST, typename T, int V, int S>
__device__ __forceinline__ void segment_maps(const Raw<T, V> (&rx)[S], const Raw<T, V> (&rr)[S], const Raw<T, V> (&ri)[S],
                                             const float (&rate)[V], int live, float (&P)[S][V], float (&H)[S][V]) {
#pragma unroll
  for (int k = 0; k < S; ++k) {
    float x[V], r[V], i[V];
    widen<T, V>(rx[k], x);
    widen<T, V>(rr[k], r);
    widen<T, V>(ri[k], i);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float a, b;
      if constexpr (FAST) {
        const float e = expm1_small(-rate[v] * sigmoid(r[v]));
        a = 1.f + e;
        const float z = fmaf(-e, e, -2.f * e), q = 1.f + __expf(-i[v]);
        b = z * rsqrt_approx(z * q * q) * x[v];
      } else {
        const Gate g = gate_any(r[v], rate[v]);
        a = g.a;
        b = g.s * sigmoid(i[v]) * x[v];
      }
      if (k >= live) a = 1.f, b = 0.f;
      P[k][v] = k == 0 ? a : a * P[k > 0 ? k - 1 : 0][v];
      H[k][v] = k == 0 ? b : fmaf(a, H[k > 0 ? k - 1 : 0][v], b);
    }
  }
}

template <typename T, int V, int S, int W, bool CL>
__global__ void __launch_bounds__(32 * W)
scan_fwd_kernel(ScanArgs s, int ns, int slabs) {
  __shared__ MapBuffers<V, W> maps;
  if constexpr (CL) cluster_arrive();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = CL ? blockIdx.x / (uint32_t)ns : blockIdx.x;
  const int rank = CL ? (int)(blockIdx.x - unit * (uint32_t)ns) : 0;
  const int64_t b = unit / (uint32_t)slabs;
  const int d = ((int)(unit - (uint32_t)b * (uint32_t)slabs) * 32 + lane) * V;
  const bool mine = d < s.D;
  const T* x = static_cast<const T*>(s.x) + b * s.sx.b + d;
  const T* r = static_cast<const T*>(s.r) + b * s.sr.b + d;
  const T* g = static_cast<const T*>(s.i) + b * s.si.b + d;
  T* y = static_cast<T*>(s.y) + b * s.sy.b + d;
  const int64_t chunks = (s.T + kChunk - 1) / kChunk;
  grid_dependency_wait();
  const int64_t n = seq_len(s.lens, b, s.T);
  float rate[V], carry[V];
  bool rates = true;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = mine ? decay_rate(s.lam[d + v], s.decay) : 0.1f;
    carry[v] = mine && s.h0 ? s.h0[b * s.D + d + v] : 0.f;
    rates = rates && fast_rate(rate[v]);
  }
  const int64_t tile = (int64_t)ns * W * S, rounds = (n + tile - 1) / tile;
  int64_t t = ((int64_t)rank * W + warp) * S;  // this warp's segment
  Raw<T, V> rx[S], rr[S], ri[S];
  ld_rows<T, V, S>(rr, r, s.sr.t, t, n, mine);
  ld_rows<T, V, S>(ri, g, s.si.t, t, n, mine);
  ld_rows<T, V, S>(rx, x, s.sx.t, t, n, mine);
  if constexpr (CL) cluster_wait();  // every block of the cluster has started: its shared memory may be written
  for (int64_t round = 0; round < rounds; ++round, t += tile) {
    float P[S][V], H[S][V], start[V];
    const int live = n - t < S ? (n > t ? (int)(n - t) : 0) : S;
    if (all_fast<T, V, S>(rr, rates))
      segment_maps<true, T, V, S>(rx, rr, ri, rate, live, P, H);
    else
      segment_maps<false, T, V, S>(rx, rr, ri, rate, live, P, H);
    ld_rows<T, V, S>(rr, r, s.sr.t, t + tile, n, mine);
    ld_rows<T, V, S>(ri, g, s.si.t, t + tile, n, mine);
    ld_rows<T, V, S>(rx, x, s.sx.t, t + tile, n, mine);
    exchange<V, W, CL, false>(maps, (int)(round & 1), warp, lane, rank, ns, P[S - 1], H[S - 1], carry, start);
    if (mine) {
      if (s.saved != nullptr) {
#pragma unroll
        for (int k = 0; k < S; k += kChunk)
          if (k < live) {
            float* to = s.saved + (b * chunks + t / kChunk + k / kChunk) * s.D + d;
#pragma unroll
            for (int v = 0; v < V; ++v) to[v] = k == 0 ? start[v] : fmaf(P[k > 0 ? k - 1 : 0][v], start[v], H[k > 0 ? k - 1 : 0][v]);
          }
      }
#pragma unroll
      for (int k = 0; k < S; ++k) {
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = k < live ? fmaf(P[k][v], start[v], H[k][v]) : 0.f;
        if (k < live || t + k < s.T) st_raw<T, V>(y + (t + k) * s.sy.t, narrow<T, V>(o));
      }
    }
  }
  if (mine) {
    if (s.hT != nullptr && rank == 0 && warp == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) s.hT[b * s.D + d + v] = carry[v];
    const float none[V] = {};
    for (; t < s.T; t += tile)
      for (int k = 0; k < S && t + k < s.T; ++k) st_raw<T, V>(y + (t + k) * s.sy.t, narrow<T, V>(none));
  }
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
  float c1[S][V], c2[S][V], c3[S][V], G[S][V], Q[S][V];
  float outp[V], outq[V];  // the map of a segment: u -> outp u + outq
  float sumG[V], sumQ[V];
};

template <bool FAST, typename T, int V, int S>
__device__ __forceinline__ void segment_factors(const Raw<T, V> (&rx)[S], const Raw<T, V> (&rr)[S],
                                                const Raw<T, V> (&ri)[S], const Raw<T, V> (&rg)[S], const float (&rate)[V],
                                                const float (&h0)[V], int live, Factors<V, S>& f) {
  float a[S][V], c4[S][V], h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = h0[v];
#pragma unroll
  for (int k = 0; k < S; ++k) {
    float x[V], r[V], i[V];
    widen<T, V>(rx[k], x);
    widen<T, V>(rr[k], r);
    widen<T, V>(ri[k], i);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Gate q = FAST ? gate_fast(r[v], rate[v]) : gate_any(r[v], rate[v]);
      const float si = sigmoid(i[v]), c1 = q.s * si, b = c1 * x[v];
      const bool on = k < live;
      a[k][v] = on ? q.a : 1.f;
      c4[k][v] = on ? q.a * fmaf(h[v], q.g, -(q.a * si) * (x[v] * q.k)) : 0.f;
      f.c1[k][v] = on ? c1 : 0.f;
      f.c2[k][v] = on ? b * (1.f - si) : 0.f;
      f.c3[k][v] = on ? -rate[v] * (1.f - q.g) * c4[k][v] : 0.f;
      h[v] = on ? fmaf(q.a, h[v], b) : h[v];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) f.sumG[v] = 0.f, f.sumQ[v] = 0.f;
#pragma unroll
  for (int k = S - 1; k >= 0; --k) {
    float dy[V];
    widen<T, V>(rg[k], dy);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = k + 1 < S ? k + 1 : k;
      f.G[k][v] = k == S - 1 ? dy[v] : fmaf(a[j][v], f.G[j][v], dy[v]);
      f.Q[k][v] = k == S - 1 ? 1.f : a[j][v] * f.Q[j][v];
      f.sumG[v] = fmaf(c4[k][v], f.G[k][v], f.sumG[v]);
      f.sumQ[v] = fmaf(c4[k][v], f.Q[k][v], f.sumQ[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) f.outp[v] = a[0][v] * f.Q[0][v], f.outq[v] = a[0][v] * f.G[0][v];
}

template <typename T, int V, int W, bool CL>
__global__ void __launch_bounds__(32 * W)
scan_bwd_kernel(ScanArgs s, int ns, int slabs) {
  constexpr int S = kChunk;
  __shared__ MapBuffers<V, W> maps;
  if constexpr (CL) cluster_arrive();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = CL ? blockIdx.x / (uint32_t)ns : blockIdx.x;
  const int rank = CL ? (int)(blockIdx.x - unit * (uint32_t)ns) : 0;
  const int64_t b = unit / (uint32_t)slabs;
  const int d = ((int)(unit - (uint32_t)b * (uint32_t)slabs) * 32 + lane) * V;
  const bool mine = d < s.D;
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
  bool rates = true;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = mine ? decay_rate(s.lam[d + v], s.decay) : 0.1f;
    carry[v] = mine && s.dhT ? s.dhT[b * s.D + d + v] : 0.f;
    dsum[v] = 0.f;
    rates = rates && fast_rate(rate[v]);
  }
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
  if constexpr (CL) cluster_wait();  // every block of the cluster has started: its shared memory may be written
  for (int64_t round = 0; round < rounds; ++round, t -= tile) {
    Factors<V, S> f;
    float u[V];
    const int live = n - t < S ? (n > t ? (int)(n - t) : 0) : S;
    if (all_fast<T, V, S>(rr, rates))
      segment_factors<true, T, V, S>(rx, rr, ri, rg, rate, h0, live, f);
    else
      segment_factors<false, T, V, S>(rx, rr, ri, rg, rate, h0, live, f);
    load(t - tile);
    exchange<V, W, CL, true>(maps, (int)(round & 1), warp, lane, rank, ns, f.outp, f.outq, carry, u);
    if (mine) {
#pragma unroll
      for (int k = 0; k < S; ++k) {
        float ox[V], orr[V], oi[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float gh = fmaf(f.Q[k][v], u[v], f.G[k][v]);
          ox[v] = f.c1[k][v] * gh, oi[v] = f.c2[k][v] * gh, orr[v] = f.c3[k][v] * gh;
        }
        if (k < live || t + k < s.T) {
          st_raw<T, V>(dx + (t + k) * s.sx.t, narrow<T, V>(ox));
          st_raw<T, V>(dr + (t + k) * s.sr.t, narrow<T, V>(orr));
          st_raw<T, V>(di + (t + k) * s.si.t, narrow<T, V>(oi));
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) dsum[v] += fmaf(f.sumQ[v], u[v], f.sumG[v]);
  }
  // the block's partial sum of dlam: its warps in order
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) maps.warp[0][warp][v][lane] = dsum[v];
  __syncthreads();
  if (warp == 0 && mine) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) sum += maps.warp[0][k][v][lane];
      s.ws[(b * ns + rank) * s.D + d + v] = sum;
      if (s.dh0 != nullptr && rank == 0) s.dh0[b * s.D + d + v] = carry[v];
    }
  }
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
template <typename K>
cudaError_t launch_scan(K kernel, int64_t blocks, int threads, int ns, const LaunchArgs& a, const ScanArgs& s, int slabs) {
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ns, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ns > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, s, ns, slabs);
}

// Blocks that share a slab: doubled while the slabs alone leave the GPU short
// of blocks and the sequence still fills a round.
int split_of(int64_t units, int64_t T, int tokens, int sms) {
  int ns = 1;
  while (ns < kMaxSplit && units * ns < 2 * sms && (int64_t)ns * tokens < T) ns *= 2;
  return ns;
}

bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Whether every row can be read two 16-bit channels at a time.
bool pairs_ok(const ScanArgs& s) {
  for (int64_t k : {s.sx.b, s.sx.t, s.sr.b, s.sr.t, s.si.b, s.si.t, s.sy.b, s.sy.t, (int64_t)s.D})
    if (k % 2 != 0) return false;
  for (const void* p : {s.x, s.r, s.i, (const void*)s.y, s.dy, (const void*)s.dx, (const void*)s.dr, (const void*)s.di})
    if (!aligned(p, 4)) return false;
  return true;
}

template <typename T, int V>
cudaError_t fwd_v(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int S = 16, W = 8;
  const int slabs = (s.D + 32 * V - 1) / (32 * V);
  const int64_t units = s.B * slabs;
  const int ns = split_of(units, s.T, S * W, dev.num_sms);
  if (ns == 1) return launch_scan(scan_fwd_kernel<T, V, S, W, false>, units, 32 * W, 1, a, s, slabs);
  return launch_scan(scan_fwd_kernel<T, V, S, W, true>, units * ns, 32 * W, ns, a, s, slabs);
}

template <typename T, int V>
cudaError_t bwd_v(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int W = 8;
  const int slabs = (s.D + 32 * V - 1) / (32 * V);
  const int64_t units = s.B * slabs;
  const int ns = split_of(units, s.T, kChunk * W, dev.num_sms);
  cudaError_t e = ns == 1 ? launch_scan(scan_bwd_kernel<T, V, W, false>, units, 32 * W, 1, a, s, slabs)
                          : launch_scan(scan_bwd_kernel<T, V, W, true>, units * ns, 32 * W, ns, a, s, slabs);
  if (e != cudaSuccess) return e;
  return launch_kernel(scan_dlam_kernel, dim3((unsigned)((s.D + 31) / 32)), dim3(32, kSumRows), 0, a,
                       (const float*)s.ws, s.B * ns, s.D, s.lam, s.decay, s.dlam);
}

template <typename T>
cudaError_t fwd(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  if (s.T == 1) {
    const int block = 128;
    return launch_kernel(scan_step_kernel<T>, dim3((unsigned)((s.B * s.D + block - 1) / block)), dim3(block), 0, a, s);
  }
  if (sizeof(T) == 2 && pairs_ok(s)) return fwd_v<T, 4 / sizeof(T)>(s, a, dev);
  return fwd_v<T, 1>(s, a, dev);
}

template <typename T>
cudaError_t bwd(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  if (sizeof(T) == 2 && pairs_ok(s)) return bwd_v<T, 4 / sizeof(T)>(s, a, dev);
  return bwd_v<T, 1>(s, a, dev);
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
