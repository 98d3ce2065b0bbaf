// 8-bit matrix product with scales for each row of both sides (gconv_matmul_q8):
//   y[m, n] = sx[m] * sw[n] * sum_k xq[m, k] * wq[n, k] (+ bias[n])
#include <algorithm>

#include "seq.h"
#include "seq_vec.cuh"

namespace gconv {
namespace {

// scales and bias in fp32, one rounding
template <typename T>
__device__ __forceinline__ float finish(float acc, float sx, float sw, float bias) {
  return fmaf(acc * sx, sw, bias);
}

// Any sizes and alignment: 64 x 64 outputs a block, 4 x 4 a thread, four
// products an instruction (signed 8-bit dot product, 32-bit integer sums).
template <typename T>
__global__ void __launch_bounds__(256) mmq_any_kernel(MatmulQ8Args a) {
  __shared__ int xs[64][17], ws[64][17];
  allow_dependent_launch();
  grid_dependency_wait();
  const int64_t m0 = (int64_t)blockIdx.x * 64;
  const int n0 = blockIdx.y * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 64) {
    for (int q = threadIdx.x; q < 64 * 16; q += 256) {
      const int row = q >> 4, col = q & 15;
      uint32_t vx = 0, vw = 0;
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + col * 4 + j;
        if (k < a.K) {
          if (m0 + row < a.M) vx |= (uint32_t)(uint8_t)a.xq[(m0 + row) * a.K + k] << (8 * j);
          if (n0 + row < a.N) vw |= (uint32_t)(uint8_t)a.wq[(int64_t)(n0 + row) * a.K + k] << (8 * j);
        }
      }
      xs[row][col] = (int)vx, ws[row][col] = (int)vw;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      int xv[4], wv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) xv[j] = xs[ty + 16 * j][c], wv[j] = ws[tx + 16 * j][c];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xv[i], wv[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty + 16 * i;
    if (m >= a.M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= a.N) continue;
      const float b = a.bias ? Elem<T>::to_f32(static_cast<const T*>(a.bias)[n]) : 0.f;
      static_cast<T*>(a.y)[m * a.ys + n] = Elem<T>::from_f32(finish<T>((float)acc[i][j], a.sx[m], a.sw[n], b));
    }
  }
}

template <typename T>
cudaError_t launch(const MatmulQ8Args& m, const LaunchArgs& a, const DeviceInfo& dev) {
  const dim3 grid((unsigned)((m.M + 63) / 64), (unsigned)((m.N + 63) / 64));
  return launch_kernel(mmq_any_kernel<T>, grid, dim3(256), 0, a, m);
}

}  // namespace

cudaError_t matmul_q8_launch(const MatmulQ8Args& m, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (a.dt) {
    case kF32: return launch<float>(m, a, dev);
    case kF16: return launch<__half>(m, a, dev);
    default: return launch<__nv_bfloat16>(m, a, dev);
  }
}

}  // namespace gconv
