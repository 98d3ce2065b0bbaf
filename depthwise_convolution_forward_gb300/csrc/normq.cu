// Residual addition + root-mean-square norm with an 8-bit output, and the row
// quantiser (gconv_rms_norm_q8, gconv_quantize_rows_q8).
//
//   h = round(x + residual);  v = h / sqrt(mean(h^2) + eps) * weight
//   scale = max|v| / 127;  q = round(v / scale)
//
// The factor 1 / sqrt(...) is the same for a whole row, so it cancels from
// v / scale: with f = h * weight, q = round(127 f / max|f|) and
// scale = max|f| / sqrt(...) / 127.  One pass over the row gives the sum of
// squares and max|f| together.
#include <algorithm>

#include "seq.h"
#include "seq_vec.cuh"

namespace gconv {
namespace {

// 127 v / m rounded to an integer, for |v| <= m; pre = 2^100 keeps 127 / m
// finite where m is tiny.
struct Quant {
  float pre, inv;
  __device__ __forceinline__ explicit Quant(float m) {
    pre = m < 1e-30f ? 0x1p100f : 1.f;
    inv = m > 0.f && m < INFINITY ? 127.f / (m * pre) : 0.f;
  }
  __device__ __forceinline__ int operator()(float v) const {
    const int q = __float2int_rn((v * pre) * inv);  // NaN gives 0
    return q < -127 ? -127 : q > 127 ? 127 : q;
  }
};

// Sum, and maximum of non-negative floats as their bit patterns (in which a
// NaN is above infinity), over a block.  Every thread gets both.
__device__ __forceinline__ void block_sum_max(float& sum, uint32_t& mx) {
  __shared__ float ssum[32];
  __shared__ uint32_t smax[32];
  const int warps = (blockDim.x + 31) / 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (warps == 1) return;
  if (lane == 0) ssum[warp] = sum, smax[warp] = mx;
  __syncthreads();
  sum = lane < warps ? ssum[lane] : 0.f;
  mx = lane < warps ? smax[lane] : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  mx = __reduce_max_sync(0xffffffffu, mx);
}

// The row's factor 1 / sqrt(mean + eps), the scale, and the quantiser's
// largest value (0: q is 0 throughout).
__device__ __forceinline__ void row_stats(const NormArgs& n, float sum, uint32_t mxbits, float* rstd, float* scale,
                                          float* m) {
  const float mx = __uint_as_float(mxbits);
  bool bad = !(mx < INFINITY);
  *rstd = 1.f;
  if (n.norm) {
    const float ms = sum / (float)n.D + n.eps;
    bad = bad || !(sum < INFINITY);
    *rstd = ms > 0.f ? rsqrtf(ms) : ms == 0.f ? 0.f : ms;
  }
  *scale = bad ? __int_as_float(0x7fffffff) : mx * *rstd / 127.f;
  *m = bad ? 0.f : mx;
}

// Any width, stride and alignment: one block for each row, the row's h in
// shared memory.
template <typename T>
__global__ void __launch_bounds__(256) norm_q8_any_kernel(NormArgs n) {
  extern __shared__ __align__(16) unsigned char smem[];
  T* hs = reinterpret_cast<T*>(smem);
  allow_dependent_launch();
  grid_dependency_wait();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(n.x) + row * n.sx;
  const T* res = n.res ? static_cast<const T*>(n.res) + row * n.sr : nullptr;
  const T* w = static_cast<const T*>(n.w);
  T* ro = n.res_out ? static_cast<T*>(n.res_out) + row * n.sr : nullptr;
  float sum = 0.f;
  uint32_t mx = 0;
  for (int k = threadIdx.x; k < n.D; k += blockDim.x) {
    T h = x[k];
    if (res) h = Elem<T>::from_f32(Elem<T>::to_f32(h) + Elem<T>::to_f32(res[k]));
    if (ro) ro[k] = h;
    hs[k] = h;
    const float f = Elem<T>::to_f32(h);
    sum = fmaf(f, f, sum);
    mx = max(mx, __float_as_uint(fabsf(w ? f * Elem<T>::to_f32(w[k]) : f)));
  }
  block_sum_max(sum, mx);
  float rstd, scale, m;
  row_stats(n, sum, mx, &rstd, &scale, &m);
  const Quant quant(m);
  for (int k = threadIdx.x; k < n.D; k += blockDim.x) {
    const float f = Elem<T>::to_f32(hs[k]), g = w ? Elem<T>::to_f32(w[k]) : 1.f;
    if (n.q) n.q[row * n.D + k] = (int8_t)quant(f * g);
    if (n.y) static_cast<T*>(n.y)[row * n.sy + k] = Elem<T>::from_f32(f * rstd * g);
  }
  if (n.scale && threadIdx.x == 0) n.scale[row] = scale;
}

template <typename T>
cudaError_t launch(const NormArgs& n, const LaunchArgs& a, const DeviceInfo& dev) {
  const size_t smem = (size_t)n.D * sizeof(T);
  cudaError_t e = cudaFuncSetAttribute(norm_q8_any_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       GCONV_NORM_MAX_D * (int)sizeof(T));
  if (e != cudaSuccess) return e;
  return launch_kernel(norm_q8_any_kernel<T>, dim3((unsigned)n.rows), dim3(256), smem, a, n);
}

}  // namespace

cudaError_t norm_q8_launch(const NormArgs& n, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (a.dt) {
    case kF32: return launch<float>(n, a, dev);
    case kF16: return launch<__half>(n, a, dev);
    default: return launch<__nv_bfloat16>(n, a, dev);
  }
}

}  // namespace gconv
