// Selective scan, backward (gconv_selective_scan_bwd).
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "plan_cache.h"
#include "sscan.cuh"

namespace gconv {
namespace {

// ---------------------------------------------------------------------------
// A block owns CC channels of a group of one sequence and walks its part of the tokens
// backwards, a saved chunk of kChunk tokens at a time: the states are walked forward again from the saved
// one and those before even tokens kept in shared memory, then g comes back through them, a pair of tokens at a time
// (the state between them from the one before).  A lane has four states of two channels.
// Per token and state, with ag = a_{t+1} g_{t+1}:
//   g = C do + ag;  dC += h do, dB += g u (over the channels);  du += g B (over the states)
//   ag' = a g;  q = ag' h_{t-1};  dA += q s;  ds += q A (over the states)
// The sums over channels are taken over a warp's lanes, then over the block's warps in shared memory, and
// left as this block's share in the workspace; a second launch adds the shares in order.
//
// PRE: where the walk is split, a first launch takes every part but the first for the g that it
// sends out when none comes in, and the sum of its steps (the fold is ag <- exp(A sum s) ag + G).
//
// Every token's B and C gradients are sums over channels, its du and ds sums over states: 12 shuffles a token and lane
// after the lane's own sums over its two channels and four states.  Eight and four channels' lanes each keep half of
// what is left: the order of a lane's states and channels is permuted by its place, so that what it keeps and what it
// sends are fixed registers.  8 x 2048 x 2048 with 16 states, bf16, gated: 730 us (the sums of the shares 21 of them),
// 1 x 32768 x 2048 1515.  50% of the issue slots at 10% of the warps (247 registers, two blocks an SM) and 54% of the
// cycles of shared memory's pipe: bound by these and by the chains of one pair of tokens.  The whole history in shared
// memory, tokens one by one and selections at every shuffle took 1076; three blocks an SM at 168 registers spilled, 1.3
// to 1.6 times as long.  Other numbers of states: 8: 587; 32 (8 x 2048 x 1024): 734; 64 (x 512): 802.
// VEC: rows of vectors.  Others are asked for by the aligned words that hold them: 8 x 2048 x 2047 950 (1145 by
// elements that were waited for); one kernel for both took 751 for the aligned rows.
// ---------------------------------------------------------------------------
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCh = 2;  // channels of a lane

template <int SL>
struct Tile {
  static constexpr int NP = kNS * SL;
  static constexpr int CL = 32 / SL;                // lanes of channels
  static constexpr int CC = kWarps * kCh * CL;
  static constexpr int VE = SL <= 4 ? 8 : 32 / SL;  // elements of a thread
  static constexpr int RT = CC / VE;                // threads of a row
  static constexpr int RP = kThreads / RT;          // rows of a pass
  static constexpr int PASSES = kChunk / RP;
  static constexpr int P = CC + 4;                  // pitch of the sums' rows
  static constexpr int PERM = CL >= 4 ? 3 : CL - 1; // lanes of channels by which a lane's states are permuted
  static constexpr int MIX = (kChunk * NP / 4 + kThreads - 1) / kThreads;  // fours of B and C a thread
  struct Buf {
    float2 su[kChunk][CC];  // step, step x; channel c of a row at c ^ (c / 8 % 8)
    float go[kChunk][CC];   // do, at the same place
    float4 b[kChunk][PERM + 1][NP / 4], c[kChunk][PERM + 1][NP / 4];  // four states in each order k ^ perm
    float du[kChunk][P], ds[kChunk][P], o[kChunk][P];
    float mix[kWarps][kChunk][2 * NP];
    float4 h[kChunk / 2][kCh][kThreads];  // the state before every other token
  };
  // A thread's own elements of the chunk that comes next, as they lie in memory.
  template <typename T, bool VEC>
  struct Ahead {
    static constexpr int kPieces = VE * (int)sizeof(T) > 16 ? 2 : 1;
    uint4 rows[4][PASSES][kPieces][kThreads];  // x, delta, z, dy
    uint4 mix[2][MIX][kThreads];               // B, C
    uint32_t rest[VEC ? 1 : 4][VEC ? 1 : PASSES][VEC ? 1 : kThreads];  // a row's word past its piece (ask_words)
  };
  struct PreBuf {
    float2 su[kChunk][CC];
    float go[kChunk][CC];
    float4 c[kChunk][PERM + 1][NP / 4];
  };
};
// V elements from p, `left` of them there, to a thread's pieces of shared memory, kThreads apart, without waiting
// where a copy fits them.  ask_words is for rows of any alignment: the aligned words that hold any of the elements are
// copied, and joined by shifts when they are read (`rest` is the place of a word past the pieces).  A row's first and
// last word may hold a half of what lies beside it: chunks with a tensor's first or last row (end_chunk), beside which
// nothing may lie, come by elements to the same places and are waited for (ask_elements; inlined, its registers would be
// every chunk's: 8 x 2048 x 2047 1013 us, so 950).
template <typename T, int V>
__device__ __forceinline__ uint32_t* word_at(uint4* to, uint32_t* rest, int k) {
  constexpr int pieces = (V * (int)sizeof(T) / 4 + 3) / 4;
  return k < 4 * pieces ? reinterpret_cast<uint32_t*>(to + k / 4 * kThreads) + k % 4 : rest;
}
template <typename T, int V>
__device__ __forceinline__ void ask_words(uint4* to, uint32_t* rest, const T* p, int left) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const int off = (int)(at & 3) / (int)sizeof(T), have = left < V ? left : V;  // elements of the first word before p
#pragma unroll
  for (int k = 0; k < V * (int)sizeof(T) / 4 + (sizeof(T) == 2 ? 1 : 0); ++k)
    if (have > 0 && k * (4 / (int)sizeof(T)) < have + off)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(word_at<T, V>(to, rest, k))),
                   "l"(reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3) + k)
                   : "memory");
}
template <typename T, int V>
__device__ __noinline__ void ask_elements(uint4* to, uint32_t* rest, const T* p, int left) {
  static_assert(sizeof(T) == 2, "a word of a wider type is an element");
  const int off = (int)(reinterpret_cast<uintptr_t>(p) & 2) / 2;
  uint16_t v[V];
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < left) v[e] = reinterpret_cast<const uint16_t*>(p)[e];
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < left) reinterpret_cast<uint16_t*>(word_at<T, V>(to, rest, (e + off) / 2))[(e + off) & 1] = v[e];
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> answer_words(const uint4* from, const uint32_t* rest, const T* p, int left) {
  constexpr int words = V * (int)sizeof(T) / 4, pieces = (words + 3) / 4;
  const int shift = (int)(reinterpret_cast<uintptr_t>(p) & 2) * 8;
  Raw<T, V> r;
  auto word = [&](int k) {
    return k < 4 * pieces ? reinterpret_cast<const uint32_t*>(from + k / 4 * kThreads)[k % 4] : *rest;
  };
#pragma unroll
  for (int k = 0; k < words; ++k) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t v = __funnelshift_r(word(k), word(k + 1), shift);
      r.w[k] = 2 * k + 1 < left ? v : 2 * k < left ? v & 0xffffu : 0u;
    } else {
      r.w[k] = k < left ? word(k) : 0u;
    }
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void ask(uint4* to, const T* p, int left, bool vec) {
  constexpr int bytes = V * (int)sizeof(T), piece = bytes < 16 ? bytes : 16;
  if (vec && left >= V) {
#pragma unroll
    for (int k = 0; k < bytes / piece; ++k) {
      const uint32_t at = smem_u32(to + k * kThreads);
      if constexpr (piece == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(reinterpret_cast<const char*>(p) + 16 * k) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(p), "n"(piece) : "memory");
    }
  } else {
    const Raw<T, V> r = ld_part<T, V>(p, left, false);
#pragma unroll
    for (int k = 0; k < Raw<T, V>::kWords; ++k) reinterpret_cast<uint32_t*>(to + k / 4 * kThreads)[k % 4] = r.w[k];
  }
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> answer(const uint4* from) {
  Raw<T, V> r;
#pragma unroll
  for (int k = 0; k < Raw<T, V>::kWords; ++k) r.w[k] = reinterpret_cast<const uint32_t*>(from + k / 4 * kThreads)[k % 4];
  return r;
}
__device__ __forceinline__ int slot_of(int c) { return c ^ ((c >> 3) & 7); }

// The workspace, in floats.  `mix` is all but all of it: a tile of 256 / lanes channels leaves 2 NP floats a token, 2
// bytes a token and channel with 16 states, 8 with 32 and 32 with 64, which are written and read once.
struct Parts {
  int64_t mix, cols, ends, sums, all;
};
inline Parts parts_of(const SsmPlan& p, int64_t B, int64_t T, int D, int N, int G) {
  Parts q;
  q.mix = 0;                                                                // [tile][B][T][2 NP]
  q.cols = p.tiles(G) * B * T * 2 * kNS * lanes_of(N);                      // [B S][D (N + 2)]: dA, dskip, dbias
  q.ends = q.cols + B * p.S * D * ((int64_t)N + 2);                         // [S - 1][B][D][N]
  q.sums = q.ends + (int64_t)(p.S - 1) * B * D * N;                         // [S - 1][B][D]
  q.all = q.sums + (int64_t)(p.S - 1) * B * D;
  return q;
}

// v[k ^ perm]
__device__ __forceinline__ void permute(float (&v)[kNS], int perm) {
  const bool one = (perm & 1) != 0, two = (perm & 2) != 0;
  const float a0 = one ? v[1] : v[0], a1 = one ? v[0] : v[1], a2 = one ? v[3] : v[2], a3 = one ? v[2] : v[3];
  v[0] = two ? a2 : a0, v[1] = two ? a3 : a1, v[2] = two ? a0 : a2, v[3] = two ? a1 : a3;
}

template <typename T, int SL, bool PRE, bool VEC>
__global__ void __launch_bounds__(kThreads) ssm_back_kernel(SsmArgs s, SsmPlan p, Parts w) {
  using L = Tile<SL>;
  constexpr int VE = L::VE, NP = L::NP;
  extern __shared__ __align__(16) unsigned char smem[];
  using Buf = typename std::conditional<PRE, typename L::PreBuf, typename L::Buf>::type;
  Buf& m = *reinterpret_cast<Buf*>(smem);
  using Ahead = typename L::template Ahead<T, VEC>;
  Ahead& next = *reinterpret_cast<Ahead*>(smem + sizeof(Buf));
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = PRE ? p.S - 1 : p.S;
  const int64_t col = blockIdx.x / parts;
  const int part = (int)(blockIdx.x - col * parts) + (PRE ? 1 : 0);
  const int64_t tiles = (int64_t)p.tpg * s.G, b = col / tiles;
  const int tile = (int)(col - b * tiles), g = tile / p.tpg, group = s.D / s.G;
  const int c0 = g * group + (tile - g * p.tpg) * L::CC, cend = (g + 1) * group;
  const int sl = lane & (SL - 1), place = lane / SL;
  // A lane's order of its two channels and four states: the sums over lanes then need no selection but for what
  // is summed, since a lane always keeps its first values and sends its later ones.
  const int turn = SL > 1 ? sl & 1 : 0, perm = place & L::PERM;
  int cl[kCh], slot[kCh], left[kCh];
  int64_t state[kCh];  // of a channel's states among the sequence's
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    cl[i] = (warp * kCh + (i ^ turn)) * L::CL + place;
    slot[i] = slot_of(cl[i]);
    left[i] = c0 + cl[i] < cend ? s.N - sl * kNS : 0;
    state[i] = left[i] > 0 ? ((int64_t)c0 + cl[i]) * s.N + sl * kNS : 0;
  }
  const int row0 = threadIdx.x / L::RT, e0 = threadIdx.x % L::RT * VE, eleft = cend - c0 - e0;
  const int64_t t0 = part * p.seg, t1 = t0 + p.seg < s.T ? t0 + p.seg : s.T;
  grid_dependency_wait();
  const int64_t n = seq_len(s.lens, b, s.T), te = n < t1 ? n : t1;
  const int64_t DN = (int64_t)s.D * s.N;

  F2 A2[kCh][2], ag[kCh][2], dA[kCh][2];
  float slow[kCh];
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    float v[kNS];
    ld_states(s.A + state[i], left[i], v);
#pragma unroll
    for (int k = 0; k < kNS; ++k) v[k] *= kLog2e;
    slow[i] = slow_step(v, left[i]);
    permute(v, perm);
    A2[i][0] = f2(v[0], v[1]), A2[i][1] = f2(v[2], v[3]);
    dA[i][0] = dA[i][1] = f2(0.f, 0.f);
    float a[kNS] = {};
    if (s.dhT && part == p.S - 1) ld_states(s.dhT + b * DN + state[i], left[i], a);
    if (!PRE && part < p.S - 1) ld_states(s.ws + w.ends + ((p.S - 2) * s.B + b) * DN + state[i], left[i], a);
    permute(a, perm);
    if (!PRE && part < p.S - 1) {  // the fold of the later parts
      for (int k = p.S - 2; k > part && left[i] > 0; --k) {
        const int64_t at = (k - 1) * s.B + b;
        float end[kNS];
        ld_states(s.ws + w.ends + at * DN + state[i], left[i], end);
        permute(end, perm);
        const float sum = s.ws[w.sums + at * s.D + c0 + cl[i]];
        const F2 a01 = fold(A2[i][0], both(sum), f2(a[0], a[1]), f2(end[0], end[1]));
        const F2 a23 = fold(A2[i][1], both(sum), f2(a[2], a[3]), f2(end[2], end[3]));
        a[0] = lo(a01), a[1] = hi(a01), a[2] = lo(a23), a[3] = hi(a23);
      }
    }
    ag[i][0] = f2(a[0], a[1]), ag[i][1] = f2(a[2], a[3]);
  }
  float total[kCh] = {}, bias[VE], skips[VE], sum_skip[VE] = {}, sum_bias[VE] = {};
#pragma unroll
  for (int e = 0; e < VE; ++e) skips[e] = !PRE && s.skip && e < eleft ? s.skip[c0 + e0 + e] : 0.f;
#pragma unroll
  for (int e = 0; e < VE; ++e) bias[e] = s.delta_bias && e < eleft ? s.delta_bias[c0 + e0 + e] : 0.f;
  const int64_t ce = c0 + e0;
  const T* px = static_cast<const T*>(s.x) + b * s.sx.b + ce;
  const T* pd = static_cast<const T*>(s.delta) + b * s.sd.b + ce;
  const T* pz = s.z ? static_cast<const T*>(s.z) + b * s.sz.b + ce : nullptr;
  const T* pg = static_cast<const T*>(s.dy) + b * s.sy.b + ce;
  const T* pb = static_cast<const T*>(s.Bm) + b * s.sb.b + (int64_t)g * s.N;
  const T* pc = static_cast<const T*>(s.Cm) + b * s.sc.b + (int64_t)g * s.N;

  const int64_t last = te > t0 ? t0 + (te - 1 - t0) / kChunk * kChunk : t0 - kChunk;
  float saved[kCh][kNS];
  auto ask_row = [&, vec = p.vec](int which, int k, const T* p, int64_t stride, int64_t at, int have, auto elements) {
    uint4* const to = &next.rows[which][k][0][threadIdx.x];
    if constexpr (VEC)
      ask<T, VE>(to, p + at * stride, have, vec);
    else if constexpr (decltype(elements)::value)
      ask_elements<T, VE>(to, &next.rest[which][k][threadIdx.x], p + at * stride, have);
    else
      ask_words<T, VE>(to, &next.rest[which][k][threadIdx.x], p + at * stride, have);
  };
  auto ask_mix = [&, mix = p.mix](int which, int k, const T* p, int have, auto elements) {
    uint4* const to = &next.mix[which][k][threadIdx.x];
    if constexpr (VEC)
      ask<T, 4>(to, p, have, mix);
    else if constexpr (decltype(elements)::value)
      ask_elements<T, 4>(to, nullptr, p, have);
    else
      ask_words<T, 4>(to, nullptr, p, have);
  };
  auto row_of = [&](int which, int k, const T* p, int64_t stride, int64_t at) -> Raw<T, VE> {
    if constexpr (VEC)
      return answer<T, VE>(&next.rows[which][k][0][threadIdx.x]);
    else
      return answer_words<T, VE>(&next.rows[which][k][0][threadIdx.x], &next.rest[which][k][threadIdx.x], p + at * stride,
                                 at < te ? eleft : 0);
  };
  auto mix_of = [&](int which, int k, const T* p, int have) -> Raw<T, 4> {
    if constexpr (VEC)
      return answer<T, 4>(&next.mix[which][k][threadIdx.x]);
    else
      return answer_words<T, 4>(&next.mix[which][k][threadIdx.x], nullptr, p, have);
  };
  // asks for the chunk at t
  auto ask_all = [&](int64_t t, auto elements) {
#pragma unroll
    for (int k = 0; k < L::PASSES; ++k) {
      const int64_t at = t + row0 + k * L::RP;
      const int have = at < te ? eleft : 0;
      if (!PRE) ask_row(0, k, px, s.sx.t, at, have, elements);
      ask_row(1, k, pd, s.sd.t, at, have, elements);
      if (pz) ask_row(2, k, pz, s.sz.t, at, have, elements);
      ask_row(3, k, pg, s.sy.t, at, have, elements);
    }
#pragma unroll
    for (int k = 0; k < L::MIX; ++k) {
      const int at = threadIdx.x + k * kThreads, r = at / (NP / 4), j = at % (NP / 4);
      const int have = at < kChunk * NP / 4 && t + r < te ? s.N - 4 * j : 0;
      if (!PRE) ask_mix(0, k, pb + (t + r) * s.sb.t + 4 * j, have, elements);
      ask_mix(1, k, pc + (t + r) * s.sc.t + 4 * j, have, elements);
    }
  };
  auto fetch = [&](int64_t t) {
    if constexpr (!VEC && sizeof(T) == 2) {
      if (end_chunk(b, t, s.B, s.T))
        ask_all(t, std::true_type{});
      else
        ask_all(t, std::false_type{});
    } else {
      ask_all(t, std::false_type{});
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if constexpr (!PRE) {
#pragma unroll
      for (int i = 0; i < kCh; ++i)
        ld_states(s.saved + (b * ((s.T + kChunk - 1) / kChunk) + t / kChunk) * DN + state[i], left[i], saved[i]);
    }
  };
  if (last >= t0) fetch(last);
  for (int64_t t = last; t >= t0; t -= kChunk) {
    Raw<T, VE> x[L::PASSES], d[L::PASSES], z[L::PASSES], gy[L::PASSES];
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int k = 0; k < L::PASSES; ++k) {
      const int64_t at = t + row0 + k * L::RP;
      x[k] = PRE ? zero_raw<T, VE>() : row_of(0, k, px, s.sx.t, at);
      d[k] = row_of(1, k, pd, s.sd.t, at);
      z[k] = pz ? row_of(2, k, pz, s.sz.t, at) : zero_raw<T, VE>();
      gy[k] = row_of(3, k, pg, s.sy.t, at);
    }
    F2 h[kCh][2];
    float steps[L::PASSES][VE], gos[L::PASSES][VE];
    if constexpr (!PRE) {
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        permute(saved[i], perm);
        h[i][0] = f2(saved[i][0], saved[i][1]), h[i][1] = f2(saved[i][2], saved[i][3]);
      }
    }
#pragma unroll
    for (int k = 0; k < L::PASSES; ++k) {
      const int row = row0 + k * L::RP;
      float fx[VE], fd[VE], fg[VE], fz[VE];
      widen<T, VE>(x[k], fx);
      widen<T, VE>(d[k], fd);
      widen<T, VE>(gy[k], fg);
      widen<T, VE>(z[k], fz);
      const bool in = t + row < te;
      // (one choice for all elements: a branch each would keep them from overlapping)
#pragma unroll
      for (int e = 0; e < VE; ++e) steps[k][e] = fd[e] + bias[e], gos[k][e] = fg[e];
      if (s.softplus) {
#pragma unroll
        for (int e = 0; e < VE; ++e) steps[k][e] = softplus(steps[k][e]);
      }
      if (pz) {
#pragma unroll
        for (int e = 0; e < VE; ++e) gos[k][e] *= fz[e] * sigmoidf(fz[e]);
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        steps[k][e] = in ? steps[k][e] : 0.f;
        m.su[row][slot_of(e0 + e)] = make_float2(steps[k][e], steps[k][e] * fx[e]);
        m.go[row][slot_of(e0 + e)] = gos[k][e];
      }
    }
#pragma unroll
    for (int k = 0; k < L::MIX; ++k) {
      const int at = threadIdx.x + k * kThreads, r = at / (NP / 4), j = at % (NP / 4);
      if (at < kChunk * NP / 4) {
        float v[kNS];
        const int have = t + r < te ? s.N - 4 * j : 0;
        widen<T, 4>(mix_of(1, k, pc + (t + r) * s.sc.t + 4 * j, have), v);
#pragma unroll
        for (int q = 0; q <= L::PERM; ++q) m.c[r][q][j] = make_float4(v[q], v[1 ^ q], v[2 ^ q], v[3 ^ q]);
        if constexpr (!PRE) {
          widen<T, 4>(mix_of(0, k, pb + (t + r) * s.sb.t + 4 * j, have), v);
#pragma unroll
          for (int q = 0; q <= L::PERM; ++q) m.b[r][q][j] = make_float4(v[q], v[1 ^ q], v[2 ^ q], v[3 ^ q]);
        }
      }
    }
    if (t > t0) fetch(t - kChunk);  // into places that this thread alone reads, and has read
    __syncthreads();
    F2 lean[kCh];
#pragma unroll
    for (int i = 0; i < kCh; ++i)  // (through a shuffle: else the choice is made anew at every use, 2% of the time)
      lean[i] = both(__shfl_sync(0xffffffffu, fabsf(m.su[0][slot[i]].x) < slow[i] ? kLean : kLeanFast, lane));
    if constexpr (PRE) {
#pragma unroll
      for (int r = kChunk - 1; r >= 0; --r) {
        F2 c01, c23;
        ld_f2x2(&m.c[r][perm][sl], c01, c23);
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          const F2 ss = both(m.su[r][slot[i]].x), gg = both(m.go[r][slot[i]]);
          total[i] += lo(ss);
          ag[i][0] = mul2(decay(ss, A2[i][0], lean[i]), fma2(c01, gg, ag[i][0]));
          ag[i][1] = mul2(decay(ss, A2[i][1], lean[i]), fma2(c23, gg, ag[i][1]));
        }
      }
      __syncthreads();
    } else {
      // The states forward again, those before even tokens kept.
#pragma unroll
      for (int r = 0; r < kChunk; ++r) {
        F2 b01, b23;
        ld_f2x2(&m.b[r][perm][sl], b01, b23);
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          if (r % 2 == 0) st_f2x2(&m.h[r / 2][i][threadIdx.x], h[i][0], h[i][1]);
          const float2 su = m.su[r][slot[i]];
          const F2 ss = both(su.x), uu = both(su.y);
          h[i][0] = fma2(decay(ss, A2[i][0], lean[i]), h[i][0], mul2(uu, b01));
          h[i][1] = fma2(decay(ss, A2[i][1], lean[i]), h[i][1], mul2(uu, b23));
        }
      }
      // Sums over the SL lanes of a channel: of du, ds and o of two channels, a lane has du or ds, and o, of its
      // first channel (two lanes: all three).
      const int second = (sl >> 1) & 1;
      float* const v_at = second ? &m.ds[0][cl[0]] : &m.du[0][cl[0]];
      const bool writes = sl < 4;
      struct Token {
        F2 ss[kCh], uu[kCh], a[kCh][2], b01, b23, c01, c23;
        float go[kCh];
      };
      auto load = [&](int r, Token& k) {
        ld_f2x2(&m.b[r][perm][sl], k.b01, k.b23);
        ld_f2x2(&m.c[r][perm][sl], k.c01, k.c23);
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          const float2 su = m.su[r][slot[i]];
          k.go[i] = m.go[r][slot[i]];
          k.ss[i] = both(su.x), k.uu[i] = both(su.y);
          k.a[i][0] = decay(k.ss[i], A2[i][0], lean[i]), k.a[i][1] = decay(k.ss[i], A2[i][1], lean[i]);
        }
      };
      // A lane's parts of a token's sums.
      struct Sums {
        float b[kNS], c[kNS], u[kCh], s[kCh], o[kCh];
      };
      // A token backwards, from the states after and before it.
      auto back = [&](const Token& k, const F2 (&past)[kCh][2], const F2 (&before)[kCh][2], Sums& to) {
        F2 vB[2], vC[2];
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          const F2 gg = both(k.go[i]);
          const F2 g01 = fma2(k.c01, gg, ag[i][0]), g23 = fma2(k.c23, gg, ag[i][1]);
          if (i == 0) {
            vC[0] = mul2(past[i][0], gg), vC[1] = mul2(past[i][1], gg);
            vB[0] = mul2(g01, k.uu[i]), vB[1] = mul2(g23, k.uu[i]);
          } else {
            vC[0] = fma2(past[i][0], gg, vC[0]), vC[1] = fma2(past[i][1], gg, vC[1]);
            vB[0] = fma2(g01, k.uu[i], vB[0]), vB[1] = fma2(g23, k.uu[i], vB[1]);
          }
          const F2 u2 = fma2(g23, k.b23, mul2(g01, k.b01)), o2 = fma2(past[i][1], k.c23, mul2(past[i][0], k.c01));
          ag[i][0] = mul2(k.a[i][0], g01), ag[i][1] = mul2(k.a[i][1], g23);
          const F2 q01 = mul2(ag[i][0], before[i][0]), q23 = mul2(ag[i][1], before[i][1]);
          dA[i][0] = fma2(q01, k.ss[i], dA[i][0]), dA[i][1] = fma2(q23, k.ss[i], dA[i][1]);
          const F2 s2 = fma2(q23, A2[i][1], mul2(q01, A2[i][0]));
          to.u[i] = lo(u2) + hi(u2), to.s[i] = lo(s2) + hi(s2), to.o[i] = lo(o2) + hi(o2);
        }
        to.b[0] = lo(vB[0]), to.b[1] = hi(vB[0]), to.b[2] = lo(vB[1]), to.b[3] = hi(vB[1]);
        to.c[0] = lo(vC[0]), to.c[1] = hi(vC[0]), to.c[2] = lo(vC[1]), to.c[3] = hi(vC[1]);
      };
      // The sums of tokens r and r + 1 over the lanes, side by side: a shuffle's way takes some 25 cycles.
      auto reduce = [&](int r, Sums (&q)[2]) {
        auto over = [&](float& keep, float send, int lanes) { keep += __shfl_xor_sync(0xffffffffu, send, lanes); };
        // of channels: states by the first two bits of the place, dB or dC by the third
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
          over(q[t2].b[0], q[t2].b[1], SL), over(q[t2].b[2], q[t2].b[3], SL);
          over(q[t2].c[0], q[t2].c[1], SL), over(q[t2].c[2], q[t2].c[3], SL);
        }
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
          over(q[t2].u[0], q[t2].u[1], 1), over(q[t2].s[0], q[t2].s[1], 1);
          over(q[t2].o[0], q[t2].o[1], 1);
        }
        if constexpr (L::CL >= 4) {
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) over(q[t2].b[0], q[t2].b[2], 2 * SL), over(q[t2].c[0], q[t2].c[2], 2 * SL);
        }
        if constexpr (SL > 2) {
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) {
            const float send = second ? q[t2].u[0] : q[t2].s[0];
            q[t2].u[0] = second ? q[t2].s[0] : q[t2].u[0];
            over(q[t2].u[0], send, 2);
            over(q[t2].o[0], q[t2].o[0], 2);
          }
#pragma unroll
          for (int lanes = 4; lanes < SL; lanes <<= 1)
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {
              over(q[t2].u[0], q[t2].u[0], lanes);
              over(q[t2].o[0], q[t2].o[0], lanes);
            }
        }
        if constexpr (L::CL >= 8) {
          const bool up = (place & 4) != 0;
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) {
            const float send = up ? q[t2].b[0] : q[t2].c[0];
            q[t2].b[0] = up ? q[t2].c[0] : q[t2].b[0];
            over(q[t2].b[0], send, 4 * SL);
#pragma unroll
            for (int o = 8; o < L::CL; o <<= 1) over(q[t2].b[0], q[t2].b[0], o * SL);
          }
        }
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
          float* const to = m.mix[warp][r + t2] + sl * kNS + perm;
          if constexpr (L::CL >= 8) {
            if (place < 8) to[(place & 4) != 0 ? NP : 0] = q[t2].b[0];
          } else {
            to[0] = q[t2].b[0], to[NP] = q[t2].c[0];
            if constexpr (L::CL == 2) to[2] = q[t2].b[2], to[NP + 2] = q[t2].c[2];
          }
          if constexpr (SL == 2) {
            m.du[r + t2][cl[0]] = q[t2].u[0], m.ds[r + t2][cl[0]] = q[t2].s[0];
            m.o[r + t2][cl[0]] = q[t2].o[0];
          } else if (writes) {
            v_at[(r + t2) * L::P] = q[t2].u[0];
            if (second == 0) m.o[r + t2][cl[0]] = q[t2].o[0];
          }
        }
      };
      Sums sums[2];
      // Tokens r + 1 and r; the sums of the pair before while this one's operands are on their way.
      auto pair = [&](int r, auto first) {
        F2 before[kCh][2], mid[kCh][2];
        Token k, k1;
        load(r, k);
        load(r + 1, k1);
#pragma unroll
        for (int i = 0; i < kCh; ++i) ld_f2x2(&m.h[r / 2][i][threadIdx.x], before[i][0], before[i][1]);
        if constexpr (!decltype(first)::value) reduce(r + 2, sums);
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          mid[i][0] = fma2(k.a[i][0], before[i][0], mul2(k.uu[i], k.b01));
          mid[i][1] = fma2(k.a[i][1], before[i][1], mul2(k.uu[i], k.b23));
        }
        back(k1, h, mid, sums[1]);
        back(k, mid, before, sums[0]);
#pragma unroll
        for (int i = 0; i < kCh; ++i) h[i][0] = before[i][0], h[i][1] = before[i][1];
      };
      pair(kChunk - 2, std::true_type{});
#pragma unroll (SL <= 2 ? 1 : 4)
      for (int r = kChunk - 4; r >= 0; r -= 2) pair(r, std::false_type{});
      reduce(0, sums);
      __syncthreads();
      for (int at = threadIdx.x; at < kChunk * 2 * NP; at += kThreads) {
        const int r = at / (2 * NP), j = at % (2 * NP);
        float sum = m.mix[0][r][j];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) sum += m.mix[k][r][j];
        if (t + r < te) s.ws[w.mix + ((tile * s.B + b) * s.T + t + r) * (2 * NP) + j] = sum;
      }
#pragma unroll
      for (int k = 0; k < L::PASSES; ++k) {
        const int row = row0 + k * L::RP;
        const int64_t at = t + row;
        const bool in = at < te;
        if (at < t1 && eleft > 0) {
          float fx[VE], fd[VE], fg[VE], fz[VE], ox[VE], od[VE], oz[VE];
          widen<T, VE>(x[k], fx);
          widen<T, VE>(d[k], fd);
          widen<T, VE>(gy[k], fg);
          widen<T, VE>(z[k], fz);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float du = m.du[row][e0 + e], ds = m.ds[row][e0 + e] * kLn2;
            ox[e] = fmaf(du, steps[k][e], gos[k][e] * skips[e]);
            od[e] = fmaf(du, fx[e], ds);
            sum_skip[e] = fmaf(gos[k][e], fx[e], sum_skip[e]);
          }
          if (s.softplus) {
#pragma unroll
            for (int e = 0; e < VE; ++e) od[e] *= sigmoidf(fd[e] + bias[e]);
          }
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            ox[e] = in ? ox[e] : 0.f, od[e] = in ? od[e] : 0.f;
            sum_bias[e] += od[e];
          }
          if (s.dz) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              const float sig = sigmoidf(fz[e]), v = fmaf(skips[e], fx[e], m.o[row][e0 + e]);
              oz[e] = in ? fg[e] * v * (sig * fmaf(fz[e], 1.f - sig, 1.f)) : 0.f;
            }
            st_part<T, VE>(static_cast<T*>(s.dz) + b * s.sz.b + at * s.sz.t + ce, oz, eleft, p.vec);
          }
          st_part<T, VE>(static_cast<T*>(s.dx) + b * s.sx.b + at * s.sx.t + ce, ox, eleft, p.vec);
          st_part<T, VE>(static_cast<T*>(s.ddelta) + b * s.sd.b + at * s.sd.t + ce, od, eleft, p.vec);
        }
      }
      __syncthreads();
    }
  }
  if constexpr (PRE) {
    const int64_t at = (int64_t)(part - 1) * s.B + b;
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      float v[kNS] = {lo(ag[i][0]), hi(ag[i][0]), lo(ag[i][1]), hi(ag[i][1])};
      permute(v, perm);
      if (left[i] > 0) st_states(s.ws + w.ends + at * DN + state[i], left[i], v);
      if (sl == 0 && c0 + cl[i] < cend) s.ws[w.sums + at * s.D + c0 + cl[i]] = total[i];
    }
  } else {
    // rows past the sequence's end that no chunk covered
    const float zeros[VE] = {};
    for (int64_t t = last + kChunk; t < t1; t += kChunk)
#pragma unroll
      for (int k = 0; k < L::PASSES; ++k) {
        const int64_t at = t + row0 + k * L::RP;
        if (at < t1 && eleft > 0) {
          st_part<T, VE>(static_cast<T*>(s.dx) + b * s.sx.b + at * s.sx.t + ce, zeros, eleft, p.vec);
          st_part<T, VE>(static_cast<T*>(s.ddelta) + b * s.sd.b + at * s.sd.t + ce, zeros, eleft, p.vec);
          if (s.dz) st_part<T, VE>(static_cast<T*>(s.dz) + b * s.sz.b + at * s.sz.t + ce, zeros, eleft, p.vec);
        }
      }
    float* cols = s.ws + w.cols + (b * p.S + part) * (DN + 2 * s.D);
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      float v[kNS] = {lo(dA[i][0]), hi(dA[i][0]), lo(dA[i][1]), hi(dA[i][1])};
      permute(v, perm);
      if (left[i] > 0) st_states(cols + state[i], left[i], v);
      float a[kNS] = {lo(ag[i][0]), hi(ag[i][0]), lo(ag[i][1]), hi(ag[i][1])};
      permute(a, perm);
      if (left[i] > 0 && s.dh0 && part == 0) st_states(s.dh0 + b * DN + state[i], left[i], a);
    }
    // dskip and dbias over the rows' threads, in order
#pragma unroll
    for (int e = 0; e < VE; ++e) m.du[row0][e0 + e] = sum_skip[e], m.ds[row0][e0 + e] = sum_bias[e];
    __syncthreads();
    for (int k = threadIdx.x; k < L::CC; k += kThreads)
      if (c0 + k < cend) {
        float a = 0.f, v = 0.f;
        for (int r = 0; r < L::RP; ++r) a += m.du[r][k], v += m.ds[r][k];
        cols[DN + c0 + k] = a;
        cols[DN + s.D + c0 + k] = v;
      }
  }
}

// The blocks' shares, added in order: the first blocks take dBm and dCm (a thread an
// element, over the tiles of its group), the others dA, dskip and dbias (over sequences and parts).
template <typename T>
__global__ void __launch_bounds__(32 * kSumRows) ssm_sum_kernel(SsmArgs s, SsmPlan p, Parts w, int64_t mix_blocks) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int threads = 32 * kSumRows;
  if (blockIdx.x < mix_blocks) {
    const int NP2 = 2 * kNS * (s.N <= 8 ? 2 : s.N <= 16 ? 4 : s.N <= 32 ? 8 : 16);
    const int64_t id = blockIdx.x * (int64_t)threads + threadIdx.y * 32 + threadIdx.x, mixes = (int64_t)s.G * s.N;
    if (id >= s.B * s.T * mixes) return;
    const int64_t bt = id / mixes, b = bt / s.T, t = bt - b * s.T;
    const int k = (int)(id - bt * mixes), g = k / s.N, n = k - g * s.N;
    float vb = 0.f, vc = 0.f;
    if (t < seq_len(s.lens, b, s.T)) {
      const float* at = s.ws + w.mix + ((int64_t)g * p.tpg * s.B * s.T + bt) * NP2 + n;
#pragma unroll 4
      for (int q = 0; q < p.tpg; ++q, at += s.B * s.T * NP2) vb += at[0], vc += at[NP2 / 2];
    }
    static_cast<T*>(s.dBm)[b * s.sb.b + t * s.sb.t + k] = Elem<T>::from_f32(vb);
    static_cast<T*>(s.dCm)[b * s.sc.b + t * s.sc.t + k] = Elem<T>::from_f32(vc);
    return;
  }
  const int64_t DN = (int64_t)s.D * s.N, n = DN + 2 * s.D, col = (blockIdx.x - mix_blocks) * 32 + threadIdx.x;
  const float v = column_sum(s.ws + w.cols, s.B * p.S, n, col);
  if (threadIdx.y != 0 || col >= n) return;
  if (col < DN)
    s.dA[col] = v;
  else if (col < DN + s.D) {
    if (s.dskip) s.dskip[col - DN] = v;
  } else if (s.dbias) {
    s.dbias[col - DN - s.D] = v;
  }
}

SsmPlan bwd_plan(int64_t B, int64_t T, int D, int N, int G) {
  SsmPlan p = {};
  p.CC = kThreads * kCh / lanes_of(N);
  p.tpg = (D / G + p.CC - 1) / p.CC;
  const int64_t blocks = B * p.tiles(G);
  cut_time(T, blocks, &p);
  return p;
}

int64_t sum_blocks(const SsmArgs& s, int64_t* mix_blocks) {
  const int64_t per = 32 * kSumRows;
  *mix_blocks = (s.B * s.T * s.G * s.N + per - 1) / per;
  return *mix_blocks + ((int64_t)s.D * (s.N + 2) + 31) / 32;
}

template <typename T, int SL, bool VEC>
cudaError_t launch_back(const SsmArgs& s, const SsmPlan& p, const LaunchArgs& a, const DeviceInfo& dev) {
  const Parts w = parts_of(p, s.B, s.T, s.D, s.N, s.G);
  constexpr size_t ahead = sizeof(typename Tile<SL>::template Ahead<T, VEC>);
  constexpr size_t smem = sizeof(typename Tile<SL>::Buf) + ahead, pre = sizeof(typename Tile<SL>::PreBuf) + ahead;
  static SmemAttr attr, attr_pre;
  cudaError_t e = attr.ensure(ssm_back_kernel<T, SL, false, VEC>, dev.device, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t cols = s.B * p.tiles(s.G);
  if (p.S > 1) {
    e = attr_pre.ensure(ssm_back_kernel<T, SL, true, VEC>, dev.device, (int)pre);
    if (e != cudaSuccess) return e;
    e = launch_kernel(ssm_back_kernel<T, SL, true, VEC>, dim3((unsigned)(cols * (p.S - 1))), dim3(kThreads), pre, a, s, p, w);
    if (e != cudaSuccess) return e;
  }
  e = launch_kernel(ssm_back_kernel<T, SL, false, VEC>, dim3((unsigned)(cols * p.S)), dim3(kThreads), smem, a, s, p, w);
  if (e != cudaSuccess) return e;
  int64_t mix_blocks;
  const int64_t blocks = sum_blocks(s, &mix_blocks);
  return launch_kernel(ssm_sum_kernel<T>, dim3((unsigned)blocks), dim3(32, kSumRows), 0, a, s, p, w, mix_blocks);
}

template <typename T, int SL>
cudaError_t launch(const SsmArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  SsmPlan p = bwd_plan(s.B, s.T, s.D, s.N, s.G);
  const SeqStride none = {0, 0};
  p.vec = vectors_ok({s.x, s.delta, s.z, s.dy, s.dx, s.ddelta, s.dz}, {s.sx, s.sd, s.z ? s.sz : none, s.sy}, s.D / s.G, s.G,
                     Tile<SL>::VE, sizeof(T));
  p.mix = vectors_ok({s.Bm, s.Cm}, {s.sb, s.sc}, s.N, s.G, 4, sizeof(T));
  return p.vec ? launch_back<T, SL, true>(s, p, a, dev) : launch_back<T, SL, false>(s, p, a, dev);
}

template <typename T>
cudaError_t launch_t(const SsmArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (lanes_of(s.N)) {
    case 2: return launch<T, 2>(s, a, dev);
    case 4: return launch<T, 4>(s, a, dev);
    case 8: return launch<T, 8>(s, a, dev);
    default: return launch<T, 16>(s, a, dev);
  }
}

}  // namespace

// Both directions' grids and the workspace stay within what 31 and 62 bits count, whatever
// the split (kMaxParts at most).
bool ssm_fits(int64_t B, int64_t T, int D, int N, int G) {
  const int sl = lanes_of(N);
  const double tiles = (double)G * (D / G / (256 / sl) + 1);
  return T < (int64_t)(kMaxParts - 1) << 30 && B * tiles * kMaxParts < 2e9 && (double)B * D * sl / 128 < 2e9 && (double)B * T * G * N / 512 + (double)D * (N + 2) / 32 < 2e9 &&
         tiles * B * T * 8 * sl + 64.0 * B * D * (2 * N + 4) < 1e17 && (double)chunks_of(T) * B * D * N < 1e17;
}

int64_t ssm_bwd_workspace_bytes(int64_t B, int64_t T, int D, int N, int G) {
  return parts_of(bwd_plan(B, T, D, N, G), B, T, D, N, G).all * 4;
}

cudaError_t ssm_bwd_launch(const SsmArgs& s, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (a.dt) {
    case kF32: return launch_t<float>(s, a, dev);
    case kF16: return launch_t<__half>(s, a, dev);
    default: return launch_t<__nv_bfloat16>(s, a, dev);
  }
}

}  // namespace gconv
