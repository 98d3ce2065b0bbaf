// Gated linear recurrence (gconv_gated_scan_fwd / _bwd).
//
//   l_t = -c softplus(lam) sig(r_t),  a_t = exp(l_t)
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sig(i_t) x_t
//
// Each channel of each sequence is its own recurrence.
#include <algorithm>

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
// One thread for each channel of each sequence, token after token.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void scan_fwd_seq_kernel(ScanArgs s) {
  allow_dependent_launch();
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (id >= s.B * s.D) return;
  const int64_t b = id / s.D;
  const int d = (int)(id - b * s.D);
  grid_dependency_wait();
  const int64_t n = seq_len(s.lens, b, s.T);
  const float rate = decay_rate(s.lam[d], s.decay);
  const T* x = static_cast<const T*>(s.x) + b * s.sx.b + d;
  const T* r = static_cast<const T*>(s.r) + b * s.sr.b + d;
  const T* g = static_cast<const T*>(s.i) + b * s.si.b + d;
  T* y = static_cast<T*>(s.y) + b * s.sy.b + d;
  float h = s.h0 ? s.h0[id] : 0.f;
  const int64_t chunks = (s.T + kChunk - 1) / kChunk;
  for (int64_t t = 0; t < s.T; ++t) {
    if (s.saved && t % kChunk == 0) s.saved[(b * chunks + t / kChunk) * s.D + d] = h;
    if (t < n) {
      const Gate q = gate_any(Elem<T>::to_f32(r[t * s.sr.t]), rate);
      h = fmaf(q.a, h, q.s * sigmoid(Elem<T>::to_f32(g[t * s.si.t])) * Elem<T>::to_f32(x[t * s.sx.t]));
      y[t * s.sy.t] = Elem<T>::from_f32(h);
    } else {
      y[t * s.sy.t] = Elem<T>::from_f32(0.f);
    }
  }
  if (s.hT) s.hT[id] = h;
}

template <typename T>
__global__ void scan_bwd_seq_kernel(ScanArgs s) {
  allow_dependent_launch();
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (id >= s.B * s.D) return;
  const int64_t b = id / s.D;
  const int d = (int)(id - b * s.D);
  grid_dependency_wait();
  const int64_t n = seq_len(s.lens, b, s.T);
  const float rate = decay_rate(s.lam[d], s.decay);
  const T* x = static_cast<const T*>(s.x) + b * s.sx.b + d;
  const T* r = static_cast<const T*>(s.r) + b * s.sr.b + d;
  const T* g = static_cast<const T*>(s.i) + b * s.si.b + d;
  const T* dy = static_cast<const T*>(s.dy) + b * s.sy.b + d;
  T* dx = static_cast<T*>(s.dx) + b * s.sx.b + d;
  T* dr = static_cast<T*>(s.dr) + b * s.sr.b + d;
  T* di = static_cast<T*>(s.di) + b * s.si.b + d;
  float gh = s.dhT ? s.dhT[id] : 0.f;  // gradient of the state that leaves token t
  float dsum = 0.f;
  const int64_t chunks = (s.T + kChunk - 1) / kChunk;
  for (int64_t c = chunks - 1; c >= 0; --c) {
    float hp[kChunk];  // state before each token of the chunk
    float h = s.saved[(b * chunks + c) * s.D + d];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      const int64_t t = c * kChunk + k;
      hp[k] = h;
      if (t < n) {
        const Gate q = gate_any(Elem<T>::to_f32(r[t * s.sr.t]), rate);
        h = fmaf(q.a, h, q.s * sigmoid(Elem<T>::to_f32(g[t * s.si.t])) * Elem<T>::to_f32(x[t * s.sx.t]));
      }
    }
#pragma unroll
    for (int k = kChunk - 1; k >= 0; --k) {
      const int64_t t = c * kChunk + k;
      if (t >= s.T) continue;
      float ox = 0.f, orr = 0.f, oi = 0.f;
      if (t < n) {
        const float xv = Elem<T>::to_f32(x[t * s.sx.t]);
        const float si = sigmoid(Elem<T>::to_f32(g[t * s.si.t]));
        const Gate q = gate_any(Elem<T>::to_f32(r[t * s.sr.t]), rate);
        gh += Elem<T>::to_f32(dy[t * s.sy.t]);
        const float gi = gh * si;
        ox = gi * q.s;
        oi = ox * xv * (1.f - si);
        const float w = q.a * fmaf(gh * hp[k], q.g, -(q.a * gi) * (xv * q.k));  // dl * sig(r)
        orr = -rate * w * (1.f - q.g);
        dsum += w;
        gh *= q.a;
      }
      dx[t * s.sx.t] = Elem<T>::from_f32(ox);
      dr[t * s.sr.t] = Elem<T>::from_f32(orr);
      di[t * s.si.t] = Elem<T>::from_f32(oi);
    }
  }
  if (s.dh0) s.dh0[id] = gh;
  s.ws[id] = dsum;
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

template <typename T>
cudaError_t fwd(const ScanArgs& s, const LaunchArgs& a) {
  const int block = 128;
  return launch_kernel(scan_fwd_seq_kernel<T>, dim3((unsigned)((s.B * s.D + block - 1) / block)), dim3(block), 0, a, s);
}

template <typename T>
cudaError_t bwd(const ScanArgs& s, const LaunchArgs& a) {
  const int block = 128;
  cudaError_t e =
      launch_kernel(scan_bwd_seq_kernel<T>, dim3((unsigned)((s.B * s.D + block - 1) / block)), dim3(block), 0, a, s);
  if (e != cudaSuccess) return e;
  return launch_kernel(scan_dlam_kernel, dim3((unsigned)((s.D + 31) / 32)), dim3(32, kSumRows), 0, a,
                       (const float*)s.ws, s.B, s.D, s.lam, s.decay, s.dlam);
}

}  // namespace

int64_t scan_saved_bytes(int64_t B, int64_t T, int D) { return B * ((T + kChunk - 1) / kChunk) * D * 4; }
int64_t scan_bwd_workspace_bytes(int64_t B, int64_t T, int D) { return B * D * 4; }

cudaError_t scan_fwd_launch(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo&) {
  switch (a.dt) {
    case kF32: return fwd<float>(s, a);
    case kF16: return fwd<__half>(s, a);
    default: return fwd<__nv_bfloat16>(s, a);
  }
}

cudaError_t scan_bwd_launch(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo&) {
  switch (a.dt) {
    case kF32: return bwd<float>(s, a);
    case kF16: return bwd<__half>(s, a);
    default: return bwd<__nv_bfloat16>(s, a);
  }
}

}  // namespace gconv
