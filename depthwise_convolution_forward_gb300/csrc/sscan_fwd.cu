// Selective scan, forward (gconv_selective_scan_fwd).
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "plan_cache.h"
#include "sscan.cuh"

namespace gconv {
namespace {

// ---------------------------------------------------------------------------
// Few tokens: SL lanes a channel, every lane its four states; a token's o is summed over
// the lanes.  64 x 1 x 2048 with 16 states, bf16, in a graph: 8.0 us for 18 MB of states and operands (2.7 at the
// rate of memory; they lie in the second-level cache), bound by the way from the first loads to the stores;
// 1 x 1 x 2048 2.8.
//
// Against the walk below, us, few / walk, by tokens (16 states, bf16):
//   64 x 2048 channels   4: 14.1 / 17     5: 15.8 / 17.7   8: 21.9 / 17.1
//   16 x 2048            4:  5.4 /  6.4   5:  5.9 /  6.4   8:  8.0 /  6.4
// and with 64 states, 4 x 4096, 8 tokens 12.5 / 9.4.
// ---------------------------------------------------------------------------
constexpr int kFewTokens = 4;

template <typename T, int SL>
__global__ void __launch_bounds__(128) ssm_few_kernel(SsmArgs s, bool mix) {
  allow_dependent_launch();
  const int sl = threadIdx.x & (SL - 1);
  const int64_t id = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) / SL, all = s.B * s.D;
  const bool live = id < all;
  const int64_t ch = live ? id : all - 1;  // a warp stays whole for its shuffles
  const int64_t b = s.B == 1 ? 0 : ch / s.D;
  const int d = (int)(ch - b * s.D), g = s.G == 1 ? 0 : d / (s.D / s.G), left = s.N - sl * kNS;
  const T* px = static_cast<const T*>(s.x) + b * s.sx.b + d;
  const T* pd = static_cast<const T*>(s.delta) + b * s.sd.b + d;
  const T* pz = s.z ? static_cast<const T*>(s.z) + b * s.sz.b + d : nullptr;
  const T* pb = static_cast<const T*>(s.Bm) + b * s.sb.b + (int64_t)g * s.N + sl * kNS;
  const T* pc = static_cast<const T*>(s.Cm) + b * s.sc.b + (int64_t)g * s.N + sl * kNS;
  T* py = static_cast<T*>(s.y) + b * s.sy.b + d;
  grid_dependency_wait();
  // everything is asked for before anything is used
  float A2[kNS], h[kNS] = {};
  if (s.h0) ld_states(s.h0 + ch * s.N + sl * kNS, left, h);
  ld_states(s.A + (int64_t)d * s.N + sl * kNS, left, A2);
  const float skip = s.skip ? s.skip[d] : 0.f, bias = s.delta_bias ? s.delta_bias[d] : 0.f;
  const int64_t n = seq_len(s.lens, b, s.T);
  Raw<T, 4> rb = ld_part<T, 4>(pb, left, mix), rc = ld_part<T, 4>(pc, left, mix);
  T rx = *px, rd = *pd, rz = pz ? *pz : rx;
#pragma unroll
  for (int k = 0; k < kNS; ++k) A2[k] *= kLog2e;
  const float slow = slow_step(A2, left);
  if (s.saved && live) st_states(s.saved + ch * s.N + sl * kNS, left, h);  // T <= kChunk: one state a sequence
  for (int64_t t = 0; t < s.T; ++t) {
    const float x = Elem<T>::to_f32(rx), v = Elem<T>::to_f32(rd) + bias, z = Elem<T>::to_f32(rz);
    float mb[kNS], mc[kNS];
    widen<T, kNS>(rb, mb);
    widen<T, kNS>(rc, mc);
    if (t + 1 < s.T) {
      pb += s.sb.t, pc += s.sc.t, px += s.sx.t, pd += s.sd.t;
      rb = ld_part<T, 4>(pb, left, mix), rc = ld_part<T, 4>(pc, left, mix), rx = *px, rd = *pd;
      if (pz) pz += s.sz.t, rz = *pz;
    }
    float out = 0.f;
    if (t < n) {
      const float step = step_of(v, s.softplus), u = step * x, lean = fabsf(step) < slow ? kLean : kLeanFast;
#pragma unroll
      for (int k = 0; k < kNS; ++k) {
        h[k] = fmaf(ex2f(fmaf(step, A2[k], lean)), h[k], u * mb[k]);
        out = fmaf(h[k], mc[k], out);
      }
      if (sl == 0) out = fmaf(skip, x, out);
    }
#pragma unroll
    for (int o = SL / 2; o > 0; o >>= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
    if (t < n && pz) out = out * (z * sigmoidf(z));
    if (sl == 0 && live) *py = Elem<T>::from_f32(t < n ? out : 0.f);
    py += s.sy.t;
  }
  if (s.hT && live) st_states(s.hT + ch * s.N + sl * kNS, left, h);
}

// ---------------------------------------------------------------------------
// The walk over time.  A block owns CC channels of a group of one sequence and walks the tokens of its
// part in tiles of TT.  A lane has NS states of two neighbouring channels, packed in pairs of the two, so
// that SL lanes share a pair of channels.  The block's threads widen a tile's rows once, with the step
// and step x of every pair, B and C in shared memory; each lane then walks the tile's tokens, and the sums over a
// pair's lanes, all of a tile's at once, go back through shared memory to the threads that hold x and z of the same
// elements.  Two tiles' buffers: one barrier a tile.
//
// Per token, channel and state an exponential, a product, two fused products and additions and half a product: at one
// warp's exponentials a clock and SM these alone take 58 us for 8 x 2048 x 2048 with 16 states (73 with those of the
// softplus and the gate), against 40 for the bytes.  Measured there, bf16, gated: 251 us (261 with the states saved), 1
// x 32768 x 2048 544 (with the first launch).  59% of the issue slots, at 11% of the warps (two blocks of four warps an
// SM, 125-160 registers, so that a lane's tile unrolls whole): bound by issue and by what an instruction waits for the
// one before it.  Sixteen lanes of one channel's states each, or sums in every token, took 294.  Other numbers of
// states: 8: 227; 32 (8 x 2048 x 1024): 224; 64 (x 512): 251.
// VEC: rows of vectors.  Others come and go by elements, in pairs that neighbouring threads have side by side, each
// in a register of its own: 8 x 2048 x 2047 333 (639 with eight neighbours a thread joined where they were asked for,
// 587 as words joined by shifts).  N = 15 takes B and C by elements: 323.
//
// PRE: where the walk is split, a first launch walks every part but the last, the first one from h0
// and the others from 0, for the state after it and the sum of its steps; a part then begins with the fold of
// those before it, h <- exp(A sum s) h + H.  It also keeps a copy of h0, which the last part may
// overwrite with hT before the first part of the second launch has begun.
// ---------------------------------------------------------------------------
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int TT = kChunk;
// Lanes of a pair of channels, and states of each: SL times NS.
inline int walk_lanes(int N) { return (N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64) / 4; }

template <int SL, int NS>
struct Tile {
  static_assert(SL <= 16, "VE would be 1: a thread stages a pair of channels by 8 bytes, which would lie off 8");
  static constexpr int NP = NS * SL;                   // states, with those past N
  static constexpr int PL = 32 / SL;                   // pairs of channels of a warp
  static constexpr int CC = 2 * kWarps * PL;
  static constexpr int VE = CC / 8 < 8 ? CC / 8 : 8;   // elements of a thread in a row
  static constexpr int RT = CC / VE;                   // threads of a row
  static constexpr int RP = kThreads / RT;             // rows of a pass
  static constexpr int PASSES = TT / RP;
  static constexpr int YP = CC + 2;                    // pitch of the sums' rows: lanes of a channel to different banks
  static constexpr int MIX = (TT * NP / 2 + kThreads - 1) / kThreads;  // pairs of B or C a thread
  struct Buf {
    float4 su[TT][CC / 2];  // two channels' steps and step x; pair p of a row at place_of(p)
    float b[TT][NP], c[TT][NP];
    float y[TT][YP];
  };
  struct Smem {
    Buf buf[2];
    float skip[CC], bias[CC];
  };
};
// A thread writes four neighbouring pairs, eight threads at once: to different banks.
__device__ __forceinline__ int place_of(int p) { return p ^ ((p >> 3) & 3); }

template <int NS>
__device__ __forceinline__ void ld_mix(const float* p, float (&v)[NS]) {
#pragma unroll
  for (int k = 0; k < NS; k += 4) {
    if constexpr (NS == 2) {
      const float2 a = *reinterpret_cast<const float2*>(p);
      v[0] = a.x, v[1] = a.y;
    } else {
      const float4 a = *reinterpret_cast<const float4*>(p + k);
      v[k] = a.x, v[k + 1] = a.y, v[k + 2] = a.z, v[k + 3] = a.w;
    }
  }
}

template <typename T, int SL, int NS, bool PRE, bool VEC>
__global__ void __launch_bounds__(kThreads) ssm_walk_kernel(SsmArgs s, SsmPlan p) {
  using L = Tile<SL, NS>;
  constexpr int VE = L::VE, NP = L::NP;
  extern __shared__ __align__(16) unsigned char smem[];
  typename L::Smem& m = *reinterpret_cast<typename L::Smem*>(smem);
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = PRE ? p.S - 1 : p.S;
  const int64_t col = blockIdx.x / parts;
  const int part = (int)(blockIdx.x - col * parts);
  const int64_t tiles = (int64_t)p.tpg * s.G, b = col / tiles;
  const int tile = (int)(col - b * tiles), g = tile / p.tpg, group = s.D / s.G;
  const int c0 = g * group + (tile - g * p.tpg) * L::CC, cend = (g + 1) * group;
  // the walking lane's states
  const int sl = lane & (SL - 1), pair = warp * L::PL + lane / SL, place = place_of(pair), n0 = sl * NS;
  const int64_t c = c0 + 2 * pair;
  const int la = c < cend ? s.N - n0 : 0, lb = c + 1 < cend ? s.N - n0 : 0;
  const int64_t own = la > 0 ? c * s.N + n0 : 0, next = lb > 0 ? own + s.N : 0;  // within a sequence's states
  // the staging thread's elements
  constexpr int STEP = VEC ? 2 : 2 * L::RT;  // between its pairs of elements
  const int row = threadIdx.x / L::RT, e0 = threadIdx.x % L::RT * (VEC ? VE : 2);
  const int eleft = cend - c0 - e0;
  const int64_t t0 = part * p.seg, t1 = t0 + p.seg < s.T ? t0 + p.seg : s.T;
  const int64_t DN = (int64_t)s.D * s.N;
  grid_dependency_wait();
  const int64_t n = seq_len(s.lens, b, s.T);
  const int len = (int)(t1 - t0), ne = n <= t0 ? 0 : n < t1 ? (int)(n - t0) : len;  // the part's tokens, and those inside

  F2 A2[NS], h[NS];
  ld_pairs(s.A + own, s.A + next, la, lb, A2);
#pragma unroll
  for (int k = 0; k < NS; ++k) A2[k] = mul2(A2[k], both(kLog2e)), h[k] = both(0.f);
  float first_A2[NS], second_A2[NS];
#pragma unroll
  for (int k = 0; k < NS; ++k) first_A2[k] = lo(A2[k]), second_A2[k] = hi(A2[k]);
  const F2 slow = f2(slow_step(first_A2, la), slow_step(second_A2, lb));
  float* const ends = s.ws;                                              // [S - 1][B][D][N]
  float* const first = ends + (int64_t)(p.S - 1) * s.B * DN;             // [B][D][N]: h0
  float* const sums = first + (p.S > 1 ? s.B * DN : 0);                  // [S - 1][B][D]
  if (part == 0 && s.h0) {
    const float* from = (PRE || p.S == 1 ? s.h0 : first) + b * DN;
    ld_pairs(from + own, from + next, la, lb, h);
    if (PRE) st_pairs(first + b * DN + own, first + b * DN + next, la, lb, h);
  }
  if (!PRE && part > 0) {
    ld_pairs(ends + b * DN + own, ends + b * DN + next, la, lb, h);
    for (int k = 1; k < part && la > 0; ++k) {
      const float* from = ends + (k * s.B + b) * DN;
      F2 end[NS];
      ld_pairs(from + own, from + next, la, lb, end);
      const float* at = sums + (k * s.B + b) * s.D + c;
      const F2 sum = f2(at[0], lb > 0 ? at[1] : 0.f);
#pragma unroll
      for (int e = 0; e < NS; ++e) h[e] = fold(A2[e], sum, h[e], end[e]);
    }
  }
  F2 total = both(0.f);
  for (int k = threadIdx.x; k < L::CC; k += kThreads) {
    const bool there = c0 + k < cend;
    m.bias[k] = there && s.delta_bias ? s.delta_bias[c0 + k] : 0.f;
    m.skip[k] = there && s.skip ? s.skip[c0 + k] : 0.f;
  }

  const T* px = static_cast<const T*>(s.x) + b * s.sx.b + (t0 + row) * s.sx.t + c0 + e0;
  const T* pd = static_cast<const T*>(s.delta) + b * s.sd.b + (t0 + row) * s.sd.t + c0 + e0;
  const T* pz = s.z ? static_cast<const T*>(s.z) + b * s.sz.b + (t0 + row) * s.sz.t + c0 + e0 : nullptr;
  T* py = static_cast<T*>(s.y) + b * s.sy.b + (t0 + row) * s.sy.t + c0 + e0;
  const int mr = threadIdx.x / (NP / 2), mn = threadIdx.x % (NP / 2) * 2;  // its pair of B and C
  const T* pb = static_cast<const T*>(s.Bm) + b * s.sb.b + (t0 + mr) * s.sb.t + (int64_t)g * s.N + mn;
  const T* pc = static_cast<const T*>(s.Cm) + b * s.sc.b + (t0 + mr) * s.sc.t + (int64_t)g * s.N + mn;
  constexpr int kMixRows = kThreads / (NP / 2);  // a thread's next pair of B and C is so many rows on

  using Row = typename std::conditional<VEC, Raw<T, VE>, Apart<T, VE>>::type;
  using Two = typename std::conditional<VEC, Raw<T, 2>, Apart<T, 2>>::type;
  // (p.vec is true wherever VEC is; as a constant here it lets the compiler move the loads to where they are waited for:
  // 1 x 32768 x 2048 579 us, against 537)
  auto row_at = [vec = p.vec](const T* p, int left) -> Row {
    if constexpr (VEC)
      return ld_part<T, VE>(p, left, vec);
    else
      return ld_apart<T, VE, STEP>(p, left);
  };
  auto two_at = [mix = p.mix](const T* p, int left) -> Two {
    if constexpr (VEC)
      return ld_part<T, 2>(p, left, mix);
    else
      return ld_apart<T, 2, 2>(p, left);
  };
  auto put = [vec = p.vec](T* p, const float(&v)[VE], int left) {
    if constexpr (VEC)
      st_part<T, VE>(p, v, left, vec);
    else
      st_apart<T, VE, STEP>(p, v, left);
  };
  Row x[L::PASSES], z[L::PASSES], d[L::PASSES], xn[L::PASSES], zn[L::PASSES];
  Two mb[L::MIX], mc[L::MIX];
  auto fetch = [&](int t) {  // the tile at t; rows past the end as zeros
#pragma unroll
    for (int k = 0; k < L::PASSES; ++k) {
      const int have = t + row + k * L::RP < ne ? eleft : 0;
      xn[k] = row_at(px + k * L::RP * s.sx.t, have);
      d[k] = row_at(pd + k * L::RP * s.sd.t, have);
      if (!PRE && pz) zn[k] = row_at(pz + k * L::RP * s.sz.t, have);
    }
#pragma unroll
    for (int k = 0; k < L::MIX; ++k) {
      const int have = mr + k * kMixRows < TT && t + mr + k * kMixRows < ne ? s.N - mn : 0;
      mb[k] = two_at(pb + k * kMixRows * s.sb.t, have);
      if (!PRE) mc[k] = two_at(pc + k * kMixRows * s.sc.t, have);
    }
    px += TT * s.sx.t, pd += TT * s.sd.t, pb += TT * s.sb.t;
    if (!PRE) pc += TT * s.sc.t;
    if (!PRE && pz) pz += TT * s.sz.t;
  };
  auto stage = [&](int t, typename L::Buf& to) {
#pragma unroll
    for (int k = 0; k < L::PASSES; ++k) {
      float fx[VE], fd[VE];
      widen<T, VE>(xn[k], fx);
      widen<T, VE>(d[k], fd);
      const bool in = t + row + k * L::RP < ne;
      // (one choice for all elements: a branch each would keep them from overlapping)
      float v[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) v[e] = fd[e] + m.bias[e0 + off_of<STEP>(e)];
      if (s.softplus) {
#pragma unroll
        for (int e = 0; e < VE; ++e) v[e] = softplus(v[e]);
      }
#pragma unroll
      for (int e = 0; e < VE; e += 2) {
        const float s0 = in ? v[e] : 0.f, s1 = in ? v[e + 1] : 0.f;
        to.su[row + k * L::RP][place_of((e0 + off_of<STEP>(e)) / 2)] = make_float4(s0, s1, s0 * fx[e], s1 * fx[e + 1]);
      }
    }
#pragma unroll
    for (int k = 0; k < L::MIX; ++k) {
      const int r = mr + k * kMixRows;
      if (r < TT) {
        float v[2];
        widen<T, 2>(mb[k], v);
        *reinterpret_cast<float2*>(&to.b[r][mn]) = make_float2(v[0], v[1]);
        if (!PRE) {
          widen<T, 2>(mc[k], v);
          *reinterpret_cast<float2*>(&to.c[r][mn]) = make_float2(v[0], v[1]);
        }
      }
    }
  };

  __syncthreads();
  if (ne > 0) {
    fetch(0);
    stage(0, m.buf[0]);
#pragma unroll
    for (int k = 0; k < L::PASSES; ++k) x[k] = xn[k], z[k] = zn[k];
  }
  __syncthreads();
  float* saved = s.saved ? s.saved + (b * ((s.T + kChunk - 1) / kChunk) + t0 / kChunk) * DN : nullptr;
  int which = 0;
  for (int t = 0; t < ne; t += TT, which ^= 1) {
    typename L::Buf& now = m.buf[which];
    if (t + TT < ne) fetch(t + TT);
    if (!PRE && saved) {
      st_pairs(saved + own, saved + next, la, lb, h);
      saved += DN;
    }
    // A lane's parts of the sums stay in registers over the tile, and are added over the lanes all at once:
    // the shuffles of one token hide those of another.
    // Three tokens are on their way through a warp: one's operands are read, the next one's exponentials
    // are taken, and the one before enters the states.
    struct {
      F2 ss, uu;
      float b[NS], c[NS];
    } in[3];
    struct {
      F2 a[NS], ub[NS];
    } mid[2];
    auto read = [&](int t) {
      auto& r = in[t % 3];
      ld_f2x2(&now.su[t][place], r.ss, r.uu);
      ld_mix(&now.b[t][n0], r.b);
      if constexpr (!PRE) ld_mix(&now.c[t][n0], r.c);
    };
    auto raise = [&](int t) {
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        mid[t % 2].a[k] = decay(in[t % 3].ss, A2[k], both(kLean));
        mid[t % 2].ub[k] = f2(lo(in[t % 3].uu) * in[t % 3].b[k], hi(in[t % 3].uu) * in[t % 3].b[k]);
      }
    };
    float o[2 * TT];
    read(0);
    // kLean for every exponential: another one that is chosen by the states would be one more register operand of each (538
    // to 559 us for 1 x 32768 x 2048; so 544).  Fast states make up for the rest at a whole tile's start; the choice is no
    // branch, which would hold the loads back.
    const float until = t + TT <= ne ? 1.f : INFINITY;
    const F2 by = f2(fabsf(lo(in[0].ss)) < until * lo(slow) ? 1.f : kTileGrowth,
                     fabsf(hi(in[0].ss)) < until * hi(slow) ? 1.f : kTileGrowth);
#pragma unroll
    for (int k = 0; k < NS; ++k) h[k] = mul2(h[k], by);
    read(1);
    raise(0);
#pragma unroll
    for (int q = 0; q < TT; ++q) {
      if (q + 2 < TT) read(q + 2);
      if (q + 1 < TT) raise(q + 1);
      float w0 = 0.f, w1 = 0.f;
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        h[k] = fma2(mid[q % 2].a[k], h[k], mid[q % 2].ub[k]);
        if constexpr (!PRE) w0 = fmaf(lo(h[k]), in[q % 3].c[k], w0), w1 = fmaf(hi(h[k]), in[q % 3].c[k], w1);
      }
      if constexpr (PRE) {
        total = add2(total, in[q % 3].ss);
      } else {
        o[2 * q] = w0, o[2 * q + 1] = w1;
      }
    }
    if constexpr (!PRE) {
      lane_sums<2 * TT, SL, 1>(o, sl);
#pragma unroll
      for (int k = 0; k < TT / SL; ++k)
        *reinterpret_cast<float2*>(&now.y[sl * (TT / SL) + k][2 * pair]) = make_float2(o[2 * k], o[2 * k + 1]);
    }
    if (t + TT < ne) stage(t + TT, m.buf[which ^ 1]);
    __syncthreads();
    if constexpr (!PRE) {
#pragma unroll
      for (int k = 0; k < L::PASSES; ++k) {
        const int r = row + k * L::RP;
        if (t + r < len && eleft > 0) {
          float out[VE], fx[VE], fz[VE];
          widen<T, VE>(x[k], fx);
          widen<T, VE>(z[k], fz);
          const bool in = t + r < ne;
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const int at = e0 + off_of<STEP>(e);
            out[e] = fmaf(m.skip[at], fx[e], now.y[r][at]);
          }
          if (pz) {
#pragma unroll
            for (int e = 0; e < VE; ++e) out[e] *= fz[e] * sigmoidf(fz[e]);
          }
#pragma unroll
          for (int e = 0; e < VE; ++e) out[e] = in ? out[e] : 0.f;
          put(py + k * L::RP * s.sy.t, out, eleft);
        }
        x[k] = xn[k], z[k] = zn[k];
      }
      py += TT * s.sy.t;
    }
  }
  if constexpr (PRE) {
    float* to = ends + (part * s.B + b) * DN;
    st_pairs(to + own, to + next, la, lb, h);
    float* at = sums + (part * s.B + b) * s.D + c;
    if (sl == 0 && la > 0) at[0] = lo(total);
    if (sl == 0 && lb > 0) at[1] = hi(total);
  } else {
    // rows past the sequence's end that no tile covered
    const float zeros[VE] = {};
    for (int t = (ne + TT - 1) / TT * TT; t < len; t += TT, py += TT * s.sy.t)
#pragma unroll
      for (int k = 0; k < L::PASSES; ++k)
        if (t + row + k * L::RP < len && eleft > 0) put(py + k * L::RP * s.sy.t, zeros, eleft);
    if (s.hT && part == p.S - 1) st_pairs(s.hT + b * DN + own, s.hT + b * DN + next, la, lb, h);
  }
}

SsmPlan fwd_plan(int64_t B, int64_t T, int D, int N, int G) {
  SsmPlan p = {};
  p.CC = 2 * kThreads / walk_lanes(N);
  p.tpg = (D / G + p.CC - 1) / p.CC;
  const int64_t blocks = B * p.tiles(G);
  cut_time(T, blocks, &p);
  return p;
}

template <typename T, int SL, int NS, bool VEC>
cudaError_t launch_walk(const SsmArgs& s, const SsmPlan& p, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr size_t smem = sizeof(typename Tile<SL, NS>::Smem);
  static SmemAttr attr, attr_pre;
  cudaError_t e = attr.ensure(ssm_walk_kernel<T, SL, NS, false, VEC>, dev.device, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t cols = s.B * p.tiles(s.G);
  if (p.S > 1) {
    e = attr_pre.ensure(ssm_walk_kernel<T, SL, NS, true, VEC>, dev.device, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_kernel(ssm_walk_kernel<T, SL, NS, true, VEC>, dim3((unsigned)(cols * (p.S - 1))), dim3(kThreads), smem, a, s, p);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(ssm_walk_kernel<T, SL, NS, false, VEC>, dim3((unsigned)(cols * p.S)), dim3(kThreads), smem, a, s, p);
}

template <typename T, int SL>
cudaError_t launch_few(const SsmArgs& s, const LaunchArgs& a) {
  const int64_t threads = s.B * s.D * SL;
  const bool mix = vectors_ok({s.Bm, s.Cm}, {s.sb, s.sc}, s.N, s.G, 4, sizeof(T));
  return launch_kernel(ssm_few_kernel<T, SL>, dim3((unsigned)((threads + 127) / 128)), dim3(128), 0, a, s, mix);
}

template <typename T, bool VEC>
cudaError_t launch_vec(const SsmArgs& s, const SsmPlan& p, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int NS = 4;
  if (s.N <= 8) return launch_walk<T, 8 / NS, NS, VEC>(s, p, a, dev);
  if (s.N <= 16) return launch_walk<T, 16 / NS, NS, VEC>(s, p, a, dev);
  if (s.N <= 32) return launch_walk<T, 32 / NS, NS, VEC>(s, p, a, dev);
  return launch_walk<T, 64 / NS, NS, VEC>(s, p, a, dev);
}

template <typename T>
cudaError_t launch_t(const SsmArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  if (s.T <= kFewTokens) switch (lanes_of(s.N)) {
      case 2: return launch_few<T, 2>(s, a);
      case 4: return launch_few<T, 4>(s, a);
      case 8: return launch_few<T, 8>(s, a);
      default: return launch_few<T, 16>(s, a);
    }
  SsmPlan p = fwd_plan(s.B, s.T, s.D, s.N, s.G);
  const SeqStride none = {0, 0};
  const int ve = p.CC / 8 < 8 ? p.CC / 8 : 8;
  p.vec = vectors_ok({s.x, s.delta, s.z, s.y}, {s.sx, s.sd, s.z ? s.sz : none, s.sy}, s.D / s.G, s.G, ve, sizeof(T));
  p.mix = vectors_ok({s.Bm, s.Cm}, {s.sb, s.sc}, s.N, s.G, 2, sizeof(T));
  return p.vec ? launch_vec<T, true>(s, p, a, dev) : launch_vec<T, false>(s, p, a, dev);
}

}  // namespace

int64_t ssm_saved_bytes(int64_t B, int64_t T, int D, int N) { return B * chunks_of(T) * D * N * 4; }

int64_t ssm_fwd_workspace_bytes(int64_t B, int64_t T, int D, int N, int G) {
  if (T <= kFewTokens) return 0;
  const int64_t S = fwd_plan(B, T, D, N, G).S;
  return S == 1 ? 0 : ((S - 1) * B * D * (N + 1) + B * D * N) * 4;
}

cudaError_t ssm_fwd_launch(const SsmArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (a.dt) {
    case kF32: return launch_t<float>(s, a, dev);
    case kF16: return launch_t<__half>(s, a, dev);
    default: return launch_t<__nv_bfloat16>(s, a, dev);
  }
}

}  // namespace gconv
