// Causal depthwise convolution along a sequence (gconv_causal_conv1d_*).
//
//   u_t = bias + sum_j w_j e_{t-(K-1)+j},  y_t = act(u_t)
//
// with e the sequence and, before it, the K - 1 carried rows.
#include <algorithm>

#include "seq.h"
#include "seq_vec.cuh"

namespace gconv {
namespace {

constexpr int kMaxK = GCONV_CONV1D_MAX_K;

__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// e at position t >= -(K - 1) of sequence b, channel d.
template <typename T>
__device__ __forceinline__ float ext(const ConvSeqArgs& c, int64_t b, int64_t t, int d) {
  if (t >= 0) return Elem<T>::to_f32(static_cast<const T*>(c.x)[b * c.sx.b + t * c.sx.t + d]);
  if (c.state_in == nullptr) return 0.f;
  return Elem<T>::to_f32(static_cast<const T*>(c.state_in)[(b * (c.K - 1) + t + c.K - 1) * c.D + d]);
}

template <typename T>
__device__ __forceinline__ float pre_act(const ConvSeqArgs& c, int64_t b, int64_t t, int d) {
  float u = c.bias ? Elem<T>::to_f32(static_cast<const T*>(c.bias)[d]) : 0.f;
  for (int j = 0; j < c.K; ++j)
    u = fmaf(ext<T>(c, b, t - (c.K - 1) + j, d), Elem<T>::to_f32(static_cast<const T*>(c.w)[(int64_t)d * c.K + j]), u);
  return u;
}

// One thread for each output; the thread of token 0 also moves the state.
template <typename T>
__global__ void conv1d_fwd_kernel(ConvSeqArgs c) {
  allow_dependent_launch();
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  grid_dependency_wait();
  if (id >= c.B * c.D) return;
  const int64_t b = id / c.D;
  const int d = (int)(id - b * c.D);
  const int64_t n = seq_len(c.lens, b, c.T);
  for (int64_t t = 0; t < c.T; ++t) {
    float u = 0.f;
    if (t < n) {
      u = pre_act<T>(c, b, t, d);
      if (c.act) u *= sigmoid(u);
    }
    static_cast<T*>(c.y)[b * c.sy.b + t * c.sy.t + d] = Elem<T>::from_f32(u);
  }
  if (c.state_out) {
    float last[kMaxK];
    for (int j = 0; j < c.K - 1; ++j) last[j] = ext<T>(c, b, n - (c.K - 1) + j, d);
    for (int j = 0; j < c.K - 1; ++j)
      static_cast<T*>(c.state_out)[(b * (c.K - 1) + j) * c.D + d] = Elem<T>::from_f32(last[j]);
  }
}

template <typename T>
__device__ __forceinline__ float grad_u(const ConvSeqArgs& c, int64_t b, int64_t t, int d, int64_t n) {
  if (t < 0 || t >= n) return 0.f;
  const float g = Elem<T>::to_f32(static_cast<const T*>(c.dy)[b * c.sy.b + t * c.sy.t + d]);
  if (!c.act) return g;
  const float u = pre_act<T>(c, b, t, d), s = sigmoid(u);
  return g * s * (1.f + u * (1.f - s));
}

// One thread for each channel of each sequence.
template <typename T>
__global__ void conv1d_bwd_kernel(ConvSeqArgs c) {
  allow_dependent_launch();
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  grid_dependency_wait();
  if (id >= c.B * c.D) return;
  const int64_t b = id / c.D;
  const int d = (int)(id - b * c.D);
  const int64_t n = seq_len(c.lens, b, c.T);
  const int K = c.K;
  float dw[kMaxK], db = 0.f;
  for (int j = 0; j < kMaxK; ++j) dw[j] = 0.f;
  for (int64_t p = -(K - 1); p < c.T; ++p) {
    float de = 0.f;
    if (p < n) {
      for (int j = 0; j < K; ++j)
        de = fmaf(Elem<T>::to_f32(static_cast<const T*>(c.w)[(int64_t)d * K + j]), grad_u<T>(c, b, p + K - 1 - j, d, n), de);
      if (c.dstate_out && p >= n - (K - 1))
        de += Elem<T>::to_f32(static_cast<const T*>(c.dstate_out)[(b * (K - 1) + p - (n - (K - 1))) * c.D + d]);
      if (p >= 0) {
        const float du = grad_u<T>(c, b, p, d, n);
        db += du;
        for (int j = 0; j < K; ++j) dw[j] = fmaf(du, ext<T>(c, b, p - (K - 1) + j, d), dw[j]);
      }
    }
    if (p >= 0)
      static_cast<T*>(c.dx)[b * c.sx.b + p * c.sx.t + d] = Elem<T>::from_f32(de);
    else if (c.dstate_in)
      static_cast<T*>(c.dstate_in)[(b * (K - 1) + p + K - 1) * c.D + d] = Elem<T>::from_f32(de);
  }
  float* ws = c.ws + b * (int64_t)(K + 1) * c.D + d;
  for (int j = 0; j < K; ++j) ws[(int64_t)j * c.D] = dw[j];
  ws[(int64_t)K * c.D] = db;
}

// dw[d][j] and dbias[d] from the partial rows [parts][K + 1][D].
template <typename T>
__global__ void __launch_bounds__(32 * kSumRows) conv1d_dw_kernel(ConvSeqArgs c, int64_t parts) {
  allow_dependent_launch();
  const int64_t n = (int64_t)(c.K + 1) * c.D, col = blockIdx.x * 32ll + threadIdx.x;
  grid_dependency_wait();
  const float sum = column_sum(c.ws, parts, n, col);
  if (threadIdx.y != 0 || col >= n) return;
  const int j = (int)(col / c.D), d = (int)(col - (int64_t)j * c.D);
  if (j < c.K)
    static_cast<T*>(c.dw)[(int64_t)d * c.K + j] = Elem<T>::from_f32(sum);
  else if (c.dbias)
    static_cast<T*>(c.dbias)[d] = Elem<T>::from_f32(sum);
}

template <typename T>
cudaError_t fwd(const ConvSeqArgs& c, const LaunchArgs& a) {
  return launch_kernel(conv1d_fwd_kernel<T>, dim3((unsigned)((c.B * c.D + 127) / 128)), dim3(128), 0, a, c);
}
template <typename T>
cudaError_t bwd(const ConvSeqArgs& c, const LaunchArgs& a) {
  cudaError_t e = launch_kernel(conv1d_bwd_kernel<T>, dim3((unsigned)((c.B * c.D + 127) / 128)), dim3(128), 0, a, c);
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)(c.K + 1) * c.D;
  return launch_kernel(conv1d_dw_kernel<T>, dim3((unsigned)((n + 31) / 32)), dim3(32, kSumRows), 0, a, c, c.B);
}

}  // namespace

int64_t conv1d_bwd_workspace_bytes(int64_t B, int64_t T, int D, int K) { return B * (K + 1) * D * 4; }

cudaError_t conv1d_fwd_launch(const ConvSeqArgs& c, const LaunchArgs& a, const DeviceInfo&) {
  switch (a.dt) {
    case kF32: return fwd<float>(c, a);
    case kF16: return fwd<__half>(c, a);
    default: return fwd<__nv_bfloat16>(c, a);
  }
}

cudaError_t conv1d_bwd_launch(const ConvSeqArgs& c, const LaunchArgs& a, const DeviceInfo&) {
  switch (a.dt) {
    case kF32: return bwd<float>(c, a);
    case kF16: return bwd<__half>(c, a);
    default: return bwd<__nv_bfloat16>(c, a);
  }
}

}  // namespace gconv
