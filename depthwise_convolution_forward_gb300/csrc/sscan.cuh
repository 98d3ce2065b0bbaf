// Shared parts of the selective scan's two directions (sscan_fwd.cu, sscan_bwd.cu).
//
//   s = softplus(delta + bias),  a = exp(s A)
//   h_t = a_t h_{t-1} + s_t x_t B_t,  o_t = sum_n h_t C_t + skip x_t
//
#pragma once

#include <algorithm>
#include <initializer_list>

#include "seq_vec.cuh"
#include "ssm.h"

namespace gconv {
namespace {

constexpr int kChunk = GCONV_SSM_CHUNK;
constexpr int kNS = 4;  // states that move together
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2f(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcpf(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ F2 ex2_2(F2 v) { return f2(ex2f(lo(v)), ex2f(hi(v))); }

// softplus(v) = max(v, 0) + log1p(t) with t = exp(-|v|), and log1p(t) = 2 atanh(r), r = t / (2 + t) <= 1/3.
// atanh(r) / r is a polynomial in r^2, fitted to 8e-9 of it, so that a step keeps its relative accuracy
// however small it is.
constexpr float kAtanh1 = 0.3333315849304199f, kAtanh2 = 0.20012454688549042f, kAtanh3 = 0.13980302214622498f,
                kAtanh4 = 0.1408916711807251f;
__device__ __forceinline__ float softplus(float v) {
  const float t = ex2f(-kLog2e * fabsf(v)), r = t * rcpf(2.f + t), q = r * r;
  float p = fmaf(q, kAtanh4, kAtanh3);
  p = fmaf(q, p, kAtanh2);
  p = fmaf(q, p, kAtanh1);
  p = fmaf(q, p, 1.f);
  return fmaf(2.f * r, p, fmaxf(v, 0.f));  // NaN comes through t
}
__device__ __forceinline__ F2 both(float v) { return f2(v, v); }
// A token's decay exp(s A), with A2 = A log2 e.  The hardware's base-2 exponential comes out low on average: by 5e-9 to
// 1.1e-8 of it where the argument lies in -0.0039 ... 0, by 2e-8 below (measured), and a state that lasts for many
// tokens adds that up.  A lean, added to the argument, makes up for it: kLean for slow states, kLeanFast for others, by
// the step of a chunk's first token.  2^lean is 1 in fp32, so that a step of 0 keeps the state to the bit.
// Errors of the last states with no lean, one of 2.5e-8 for all, and these, fp32, whole walks, A = -0.5 ... -1.5:
//   steps 0.0003, 6000 tokens   1.0e-5   1.9e-5   1.8e-6      steps 0.01, 1000 tokens   1.9e-6   7.8e-7   7.3e-7
//   steps 0.001, 6000           4.2e-6   9.8e-6   1.4e-6      steps 0.03, 1000          8.5e-7   4.0e-7   4.2e-7
constexpr float kLean = 9e-9f, kLeanFast = 3e-8f;
constexpr float kSlow = 0.0039f;               // the argument's magnitude from which on kLean is too little
constexpr float kTileGrowth = 1.f + 0x1p-22f;  // (kLeanFast - kLean) ln 2 of kChunk tokens
__device__ __forceinline__ F2 decay(F2 s, F2 A2, F2 lean) { return ex2_2(fma2(s, A2, lean)); }
// The step below which a lane's states, `left` of M, are slow: by the slowest of them, since a fast lean on a slow state
// is the larger error of the two.
template <int M>
__device__ __forceinline__ float slow_step(const float (&A2)[M], int left) {
  float least = INFINITY;
#pragma unroll
  for (int k = 0; k < M; ++k) least = k < left ? fminf(least, fabsf(A2[k])) : least;
  return kSlow * rcpf(least);
}
// end + exp(A sum) h, over a part's tokens whose steps add up to `sum`.  The exponential alone may leave fp32's range
// where its product with h does not (growing states; an h of 0 or near it): it enters as two equal factors.
__device__ __forceinline__ F2 fold(F2 A2, F2 sum, F2 h, F2 end) {
  const F2 half = mul2(A2, mul2(sum, both(0.5f)));
  auto most = [](float v) { return v > 127.f ? 127.f : v; };  // NaN stays
  const F2 a = ex2_2(f2(most(lo(half)), most(hi(half))));
  return fma2(a, mul2(a, h), end);
}
__device__ __forceinline__ float step_of(float v, bool soft) { return soft ? softplus(v) : v; }
__device__ __forceinline__ float sigmoidf(float v) { return rcpf(1.f + ex2f(-kLog2e * v)); }
// VE elements of a row from p, `left` of which are the row's; the rest come as zeros.
template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> ld_part(const T* p, int left, bool vec) {
  if (vec && left >= VE) return ld_raw<T, VE>(p);
  Raw<T, VE> r = zero_raw<T, VE>();
#pragma unroll
  for (int e = 0; e < VE; ++e)
    if (e < left) {
      if constexpr (sizeof(T) == 4)
        r.w[e] = reinterpret_cast<const uint32_t*>(p)[e];
      else
        r.w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
    }
  return r;
}
// The same for rows that vectors do not fit, with every element apart (joining two 16-bit ones would wait for them
// where they are asked for), in pairs that are STEP apart: element e is at off_of(e).
template <int STEP>
__device__ __forceinline__ constexpr int off_of(int e) { return e / 2 * STEP + (e & 1); }
template <typename T, int VE>
struct Apart {
  T e[VE];
};
template <typename T, int VE, int STEP>
__device__ __forceinline__ Apart<T, VE> ld_apart(const T* p, int left) {
  Apart<T, VE> r;
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    r.e[e] = Elem<T>::from_f32(0.f);
    if (off_of<STEP>(e) < left) r.e[e] = p[off_of<STEP>(e)];
  }
  return r;
}
template <typename T, int VE, int STEP>
__device__ __forceinline__ void st_apart(T* p, const float (&f)[VE], int left) {
#pragma unroll
  for (int e = 0; e < VE; ++e)
    if (off_of<STEP>(e) < left) p[off_of<STEP>(e)] = Elem<T>::from_f32(f[e]);
}
template <typename T, int VE>
__device__ __forceinline__ void widen(const Apart<T, VE>& r, float (&f)[VE]) {
#pragma unroll
  for (int e = 0; e < VE; ++e) f[e] = Elem<T>::to_f32(r.e[e]);
}
template <typename T, int VE>
__device__ __forceinline__ void st_part(T* p, const float (&f)[VE], int left, bool vec) {
  if (vec && left >= VE) {
    st_raw<T, VE>(p, narrow<T, VE>(f));
    return;
  }
#pragma unroll
  for (int e = 0; e < VE; ++e)
    if (e < left) p[e] = Elem<T>::from_f32(f[e]);
}

// Sums over LANES lanes that are STRIDE apart of NV values each, as a transposing
// butterfly: afterwards a lane whose place among them is l has, in v[0 ... NV / LANES - 1] (one
// value for NV <= LANES), the sums of the values
//   l (NV / LANES) ...                 for NV >= LANES
//   l / (LANES / NV)                   else
// NV - NV / LANES shuffles (and log2(LANES / NV) more).
template <int NV, int LANES, int STRIDE>
__device__ __forceinline__ void lane_sums(float (&v)[NV], int place) {
  int have = NV;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    if (have > 1) {
      const bool up = (place & o) != 0;
      have >>= 1;
#pragma unroll
      for (int k = 0; k < NV / 2; ++k)
        if (k < have) {
          const float keep = up ? v[k + have] : v[k], send = up ? v[k] : v[k + have];
          v[k] = keep + __shfl_xor_sync(0xffffffffu, send, o * STRIDE);
        }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o * STRIDE);
    }
  }
}

// Four floats of shared memory as two packed pairs, and back.
__device__ __forceinline__ void ld_f2x2(const float4* p, F2& a, F2& b) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
  a = v.x, b = v.y;
}
__device__ __forceinline__ void st_f2x2(float4* p, F2 a, F2 b) { *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(a, b); }

// M (2 or 4) states of a channel at p, `left` of them there.
template <int M>
__device__ __forceinline__ void ld_states(const float* p, int left, float (&h)[M]) {
  if (left >= M && (reinterpret_cast<uintptr_t>(p) & (4 * M - 1)) == 0) {
    if constexpr (M == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p);
      h[0] = v.x, h[1] = v.y;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < M; ++k) h[k] = k < left ? p[k] : 0.f;
}
template <int M>
__device__ __forceinline__ void st_states(float* p, int left, const float (&h)[M]) {
  if (left >= M && (reinterpret_cast<uintptr_t>(p) & (4 * M - 1)) == 0) {
    if constexpr (M == 4)
      *reinterpret_cast<float4*>(p) = make_float4(h[0], h[1], h[2], h[3]);
    else
      *reinterpret_cast<float2*>(p) = make_float2(h[0], h[1]);
    return;
  }
#pragma unroll
  for (int k = 0; k < M; ++k)
    if (k < left) p[k] = h[k];
}
// N states of two channels, as pairs of the two, from or to their rows a and b (la, lb of them there).
template <int N>
__device__ __forceinline__ void ld_pairs(const float* a, const float* b, int la, int lb, F2 (&h)[N]) {
  constexpr int M = N < 4 ? N : 4;
#pragma unroll
  for (int k = 0; k < N; k += M) {
    float u[M], v[M];
    ld_states<M>(a + k, la - k, u);
    ld_states<M>(b + k, lb - k, v);
#pragma unroll
    for (int e = 0; e < M; ++e) h[k + e] = f2(u[e], v[e]);
  }
}
template <int N>
__device__ __forceinline__ void st_pairs(float* a, float* b, int la, int lb, const F2 (&h)[N]) {
  constexpr int M = N < 4 ? N : 4;
#pragma unroll
  for (int k = 0; k < N; k += M) {
    float u[M], v[M];
#pragma unroll
    for (int e = 0; e < M; ++e) u[e] = lo(h[k + e]), v[e] = hi(h[k + e]);
    st_states<M>(a + k, la - k, u);
    st_states<M>(b + k, lb - k, v);
  }
}

// How a direction is cut: tiles of channels within a group, and S parts of `seg`
// tokens each of the walk over time.
struct SsmPlan {
  int CC;    // channels of a block
  int tpg;   // tiles of a group
  int S;
  int64_t seg;
  bool vec;  // rows of x, delta, z, y (and dy, ...) by vectors
  bool mix;  // rows of B and C by pairs
  int64_t tiles(int G) const { return (int64_t)tpg * G; }
};

// Whether the chunk of sequence b at token t holds a tensor's first or last row.
__host__ __device__ constexpr bool end_chunk(int64_t b, int64_t t, int64_t B, int64_t T) {
  return (b == 0 && t == 0) || (b + 1 == B && t + kChunk >= T);
}

inline int lanes_of(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
inline int64_t chunks_of(int64_t T) { return (T + kChunk - 1) / kChunk; }

// The walk is split where the blocks of whole walks are fewer than the SMs, for four blocks an SM: a part's start
// costs a first walk over the parts before it.  Forward / backward, us, by the blocks wanted (152, 304, 608, 1216):
//   1 x 32768 x 2048 bf16 (32 blocks)       1527 / 3736  1004 / 1802   544 / 1517   549 / 1565
//   2 x 8192 x 1024 f16 (32)                 320 / 931    238 / 472    147 / 423    159 / 471
//   3 x 1537 x 700 fp32 (66)                  91 / 245     62 / 135     54 / 129     54 / 129
//   8 x 2048 x 2048 bf16 (256), not split    251 / 730;  in 2 and 4 parts 356 / 868, 262 / 788
// Parts follow T, not the sequences' lengths: those past a short sequence's end have nothing to do.
// The parts' lengths are multiples of 32 tokens: of every tile and of the saved states' distance.
constexpr int kMaxParts = 64;
constexpr int kLeastPart = 64;  // tokens
inline void cut_time(int64_t T, int64_t blocks, SsmPlan* p) {
  int64_t S = blocks >= kDefaultSms ? 1 : 4 * kDefaultSms / blocks;
  S = std::min<int64_t>(S, kMaxParts);
  S = std::min(S, std::max<int64_t>(T / kLeastPart, 1));
  S = std::max<int64_t>(S, (T >> 30) + 1);  // a part's tokens are counted in 32 bits
  p->seg = ((T + S - 1) / S + 31) / 32 * 32;
  p->S = (int)((T + p->seg - 1) / p->seg);
}

inline bool vectors_ok(std::initializer_list<const void*> ps, std::initializer_list<SeqStride> st, int group, int G, int ve, int es) {
  const int bytes = ve * es < 16 ? ve * es : 16;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) return false;
  for (const SeqStride& s : st)
    if (s.b % ve != 0 || s.t % ve != 0) return false;
  return G == 1 || group % ve == 0;
}

}  // namespace
}  // namespace gconv
