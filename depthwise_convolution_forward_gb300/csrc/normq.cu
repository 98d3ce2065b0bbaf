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
#include <initializer_list>
#include <type_traits>

#include "plan_cache.h"
#include "seq.h"
#include "seq_vec.cuh"

namespace gconv {
namespace {

// 127 v / m to the nearest integer, ties to even, for |v| <= m.
//
// v * fl(127 / m) is off by up to 7.6e-6, which decides wrongly within that distance of
// a tie, and 16-bit rows are full of exact ties (every v of m / 2 is 63.5).  So the sum
// b = v inv + 1.5 * 2^23, an integer q in its low bits, is corrected by the quotient's
// distance from q: 127 / m = hi + low with hi of 10 bits, v hi - q is exact for v of up
// to 16 bits (a product of two bf16 values, or an f16 value), adding v low rounds once, and
// that is 1/2 itself at a tie, so that b plus it is rounded to nearest even.  For longer
// v the two roundings are 2^-25 together, and a tie may be missed by that.
// The one FMA alone took 72.4 us (16384 x 4096 f16), 68.6 (bf16), 48.3 (rows of bf16 as
// they are); with the distance 71.6, 70.9, 52.2; a distance that is exact for all types,
// from the remainder 127 v - q m, 78.7, 73.1, 56.0.
// pre = 2^100 or 2^-100 keeps the factors in range where m is tiny or huge.
struct Quant {
  float pre, inv, hi, low;
  static constexpr float kMagic = 12582912.f;
  __device__ __forceinline__ explicit Quant(float m) {
    pre = m < 1e-30f ? 0x1p100f : m > 1e30f ? 0x1p-100f : 1.f;
    inv = hi = low = 0.f;
    if (m > 0.f && m < INFINITY) {
      const float top = m * pre;
      inv = __fdividef(127.f, top);
      hi = __uint_as_float((__float_as_uint(inv) + 0x2000u) & ~0x3fffu);
      // (127 - hi top) / top: a product with about 1 / top, and what that missed
      const float rest = fmaf(-hi, top, 127.f), over = inv * (1.f / 127.f), about = rest * over;
      low = fmaf(fmaf(-about, top, rest), over, about);
    }
  }
  // of v pre, in the low bits of the result
  __device__ __forceinline__ float operator()(float v) const {
    const float b = fmaf(v, inv, kMagic);
    return b + fmaf(v, low, fmaf(v, hi, kMagic - b));
  }
};
// The same of two values.
__device__ __forceinline__ F2 quantise2(const Quant& q, F2 v) {
  const F2 magic = f2(Quant::kMagic, Quant::kMagic), b = fma2(v, f2(q.inv, q.inv), magic);
  const F2 d = fma2(v, f2(q.hi, q.hi), fma2(b, f2(-1.f, -1.f), magic));
  return add2(b, fma2(v, f2(q.low, q.low), d));
}

// Sum, and maximum of non-negative floats as their bit patterns (in which a
// NaN is above infinity), over a block.  Every thread gets both.
__device__ __forceinline__ void warp_sum_max(float& sum, uint32_t& mx) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  mx = __reduce_max_sync(0xffffffffu, mx);
}
__device__ __forceinline__ void block_sum_max(float& sum, uint32_t& mx) {
  __shared__ float ssum[32];
  __shared__ uint32_t smax[32];
  const int warps = (blockDim.x + 31) / 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  warp_sum_max(sum, mx);
  if (lane == 0) ssum[warp] = sum, smax[warp] = mx;
  __syncthreads();
  sum = lane < warps ? ssum[lane] : 0.f;
  mx = lane < warps ? smax[lane] : 0u;
  warp_sum_max(sum, mx);
}

// Rows whose squares come near the smallest fp32 numbers: such a row is multiplied by
// 2^100, which is exact in fp32 and bf16, and its sum and maximum are taken again; v,
// scale and q come out of them with a factor that is smaller by as much.  (Above kTiny
// what the squares lose is below 2^-24 of their sum.  f16 has no such rows but those of
// zeros.)
constexpr float kTiny = 0x1p-110f, kLift = 0x1p100f;
template <typename T>
__device__ __forceinline__ bool lifted(const NormArgs& n, float sum) {
  return !std::is_same<T, __half>::value && n.norm && sum < kTiny;
}

// The row's factor 1 / sqrt(mean + eps) from the sum as it was first (small) and as it
// is, the scale, and the quantiser's largest value (0: q is 0 throughout).
__device__ __forceinline__ void row_stats(const NormArgs& n, float first, float sum, bool lift, uint32_t mxbits, float* rstd,
                                          float* scale, float* m) {
  const float mx = __uint_as_float(mxbits);
  bool bad = !(mx < INFINITY);
  *rstd = 1.f;
  if (n.norm) {
    const bool both = lift && n.eps < kTiny;  // eps is lifted, too, where it is as small; else the sum is lost in it
    const float ms = both ? sum / (float)n.D + n.eps * kLift * kLift : first / (float)n.D + n.eps;
    bad = bad || !(sum < INFINITY);
    *rstd = ms > 0.f ? rsqrtf(ms) : ms == 0.f ? 0.f : ms;
    if (lift && !both) *rstd *= 1.f / kLift;
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
  const float first = sum;
  const bool lift = lifted<T>(n, sum);
  if (lift) {  // the whole block
    sum = 0.f, mx = 0;
    for (int k = threadIdx.x; k < n.D; k += blockDim.x) {
      const float f = Elem<T>::to_f32(hs[k]) * kLift;
      hs[k] = Elem<T>::from_f32(f);
      sum = fmaf(f, f, sum);
      mx = max(mx, __float_as_uint(fabsf(w ? f * Elem<T>::to_f32(w[k]) : f)));
    }
    __syncthreads();  // the first sums have been read
    block_sum_max(sum, mx);
  }
  float rstd, scale, m;
  row_stats(n, first, sum, lift, mx, &rstd, &scale, &m);
  const Quant quant(m);
  for (int k = threadIdx.x; k < n.D; k += blockDim.x) {
    const float f = Elem<T>::to_f32(hs[k]), g = w ? Elem<T>::to_f32(w[k]) : 1.f;
    if (n.q) n.q[row * n.D + k] = m > 0.f ? (int8_t)__float_as_uint(quant(f * g * quant.pre)) : (int8_t)0;
    if (n.y) static_cast<T*>(n.y)[row * n.sy + k] = Elem<T>::from_f32(f * rstd * g);
  }
  if (n.scale && threadIdx.x == 0) n.scale[row] = scale;
}

// 16-byte vectors: a thread keeps NV of them of its block's row in registers
// (as stored: the norm reads h rounded), so the row is read once.
template <typename T, int V>
__device__ __forceinline__ void quantise(const float (&f)[V], const Quant& quant, uint32_t (&out)[V / 4]) {
#pragma unroll
  for (int k = 0; k < V / 4; ++k) {
    const F2 a = quantise2(quant, f2(f[4 * k], f[4 * k + 1])), b = quantise2(quant, f2(f[4 * k + 2], f[4 * k + 3]));
    out[k] = __byte_perm(__byte_perm(__float_as_uint(lo(a)), __float_as_uint(hi(a)), 0x0040),
                         __byte_perm(__float_as_uint(lo(b)), __float_as_uint(hi(b)), 0x0040), 0x5410);
  }
}

// WARP: a row is a warp's, kRowWarps of them in a block.
constexpr int kRowWarps = 4;
template <typename T, int NV, bool WARP>
__global__ void __launch_bounds__(512) norm_q8_vec_kernel(NormArgs n) {
  constexpr int V = 16 / sizeof(T);
  allow_dependent_launch();
  const int threads = WARP ? 32 : (int)blockDim.x, self = WARP ? (int)threadIdx.x & 31 : (int)threadIdx.x;
  const int64_t row = WARP ? blockIdx.x * (int64_t)kRowWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (WARP && row >= n.rows) return;
  const T* x = static_cast<const T*>(n.x) + row * n.sx;
  const T* res = n.res ? static_cast<const T*>(n.res) + row * n.sr : nullptr;
  const T* w = static_cast<const T*>(n.w);
  T* ro = n.res_out ? static_cast<T*>(n.res_out) + row * n.sr : nullptr;
  grid_dependency_wait();
  Raw<T, V> h[NV], r[NV], g[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = (k * threads + self) * V;
    const bool in = e < n.D;
    h[k] = in ? ld_raw<T, V>(x + e) : zero_raw<T, V>();
    r[k] = in && res ? ld_raw<T, V>(res + e) : zero_raw<T, V>();
    g[k] = in && w ? ld_raw<T, V>(w + e) : zero_raw<T, V>();
  }
  float sum = 0.f;
  uint32_t mx = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = (k * threads + self) * V;
    float f[V];
    widen<T, V>(h[k], f);
    if (res) {
      float o[V];
      widen<T, V>(r[k], o);
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] += o[v];
      h[k] = narrow<T, V>(f);
      widen<T, V>(h[k], f);
    }
    if (ro && e < n.D) st_raw<T, V>(ro + e, h[k]);
    float gf[V];
    widen<T, V>(g[k], gf);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      sum = fmaf(f[v], f[v], sum);
      const uint32_t b = __float_as_uint(w ? f[v] * gf[v] : f[v]) & 0x7fffffffu;
      mx = b > mx ? b : mx;
    }
  }
  if constexpr (WARP)
    warp_sum_max(sum, mx);
  else
    block_sum_max(sum, mx);
  const float first = sum;
  const bool lift = lifted<T>(n, sum);
  if (lift) {  // the whole warp or block
    sum = 0.f, mx = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float f[V], gf[V];
      widen<T, V>(h[k], f);
      widen<T, V>(g[k], gf);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f[v] *= kLift;
        sum = fmaf(f[v], f[v], sum);
        mx = max(mx, __float_as_uint(w ? f[v] * gf[v] : f[v]) & 0x7fffffffu);
      }
      h[k] = narrow<T, V>(f);
    }
    if constexpr (WARP) {
      warp_sum_max(sum, mx);
    } else {
      __syncthreads();  // the first sums have been read
      block_sum_max(sum, mx);
    }
  }
  float rstd, scale, m;
  row_stats(n, first, sum, lift, mx, &rstd, &scale, &m);
  const Quant quant(m);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = (k * threads + self) * V;
    if (e >= n.D) continue;
    float f[V], gf[V];
    widen<T, V>(h[k], f);
    widen<T, V>(g[k], gf);
    if (n.y) {
      float y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = w ? f[v] * rstd * gf[v] : f[v] * rstd;
      st_raw<T, V>(static_cast<T*>(n.y) + row * n.sy + e, narrow<T, V>(y));
    }
    if (n.q) {
      uint32_t q[V / 4];
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = w ? f[v] * gf[v] : f[v];
      if (quant.pre != 1.f) {  // tiny or huge rows
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] *= quant.pre;
      }
      quantise<T, V>(f, quant, q);
#pragma unroll
      for (int v = 0; v < V / 4; ++v)
        if (m == 0.f) q[v] = 0;  // zeros, or no finite scale
      int8_t* to = n.q + row * n.D + e;
      if constexpr (V == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(q[0], q[1]);
      else
        *reinterpret_cast<uint32_t*>(to) = q[0];
    }
  }
  if (n.scale && self == 0) n.scale[row] = scale;
}

bool vectors_ok(const NormArgs& n, int V, int es) {
  for (int64_t s : {n.sx, n.res ? n.sr : 0, n.res_out ? n.sr : 0, n.y ? n.sy : 0, (int64_t)n.D})
    if (s % V != 0) return false;
  for (const void* p : {n.x, n.res, n.w, (const void*)n.res_out, (const void*)n.y})
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return (reinterpret_cast<uintptr_t>(n.q) & (V - 1)) == 0;
}

template <typename T>
cudaError_t launch(const NormArgs& n, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int V = 16 / sizeof(T);
  if (vectors_ok(n, V, sizeof(T)) && n.D <= 512 * 4 * V) {
    // Few rows: one vector a thread, the shortest way through a row (16 x 2048: below
    // the launch itself).  Many: a row in one warp where four vectors a lane
    // hold it (65536 x 512 bf16: 39.2 us, 6.0 TB/s; a block of one warp a row 67), else four
    // vectors a thread, so that a row's reductions cost fewer warps (16384 x 4096
    // f16: 71.6 us, 6.6 TB/s).
    const int vectors = n.D / V;
    const dim3 grid((unsigned)n.rows), warps((unsigned)((n.rows + kRowWarps - 1) / kRowWarps));
    auto threads = [&](int nv) { return ((vectors + nv - 1) / nv + 31) / 32 * 32; };
    if (threads(1) <= 512 && n.rows < 4 * dev.num_sms)
      return launch_kernel(norm_q8_vec_kernel<T, 1, false>, grid, dim3(threads(1)), 0, a, n);
    if (vectors <= 32) return launch_kernel(norm_q8_vec_kernel<T, 1, true>, warps, dim3(32 * kRowWarps), 0, a, n);
    if (vectors <= 64) return launch_kernel(norm_q8_vec_kernel<T, 2, true>, warps, dim3(32 * kRowWarps), 0, a, n);
    if (vectors <= 128) return launch_kernel(norm_q8_vec_kernel<T, 4, true>, warps, dim3(32 * kRowWarps), 0, a, n);
    return launch_kernel(norm_q8_vec_kernel<T, 4, false>, grid, dim3(threads(4)), 0, a, n);
  }
  const size_t smem = (size_t)n.D * sizeof(T);
  if (smem > 47 * 1024) {  // 48 KB less the reductions' few bytes is there without asking
    static SmemAttr attr;
    const cudaError_t e = attr.ensure(norm_q8_any_kernel<T>, dev.device, (int)smem);
    if (e != cudaSuccess) return e;
  }
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
