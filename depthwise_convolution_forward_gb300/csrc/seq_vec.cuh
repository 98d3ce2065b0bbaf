// Loads and stores of V consecutive channels, their widening, and packed fp32
// arithmetic for the sequence kernels.
#pragma once

#include "common.cuh"

namespace gconv {

// V elements of T as they lie in memory: one access of V * sizeof(T) bytes
// (two of 16 bytes for 32), aligned to that many.
template <typename T, int V>
struct Raw {
  static constexpr int kBytes = V * (int)sizeof(T);
  static constexpr int kWords = kBytes / 4 > 0 ? kBytes / 4 : 1;
  uint32_t w[kWords];
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> ld_raw(const T* p) {
  Raw<T, V> r;
  constexpr int bytes = Raw<T, V>::kBytes;
  if constexpr (bytes == 2) {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (bytes == 4) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (bytes == 8) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    r.w[0] = u.x, r.w[1] = u.y;
  } else {
#pragma unroll
    for (int k = 0; k < bytes / 16; ++k) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[k];
      r.w[4 * k] = u.x, r.w[4 * k + 1] = u.y, r.w[4 * k + 2] = u.z, r.w[4 * k + 3] = u.w;
    }
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void st_raw(T* p, const Raw<T, V>& r) {
  constexpr int bytes = Raw<T, V>::kBytes;
  if constexpr (bytes == 2) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)r.w[0];
  } else if constexpr (bytes == 4) {
    *reinterpret_cast<uint32_t*>(p) = r.w[0];
  } else if constexpr (bytes == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
  } else {
#pragma unroll
    for (int k = 0; k < bytes / 16; ++k)
      reinterpret_cast<uint4*>(p)[k] = make_uint4(r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]);
  }
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> zero_raw() {
  Raw<T, V> r;
#pragma unroll
  for (int k = 0; k < Raw<T, V>::kWords; ++k) r.w[k] = 0;
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void widen(const Raw<T, V>& r, float (&f)[V]) {
  if constexpr (Raw<T, V>::kBytes == 2) {
    f[0] = Elem<T>::to_f32(*reinterpret_cast<const T*>(&r.w[0]));
  } else {
    constexpr int per = 4 / (int)sizeof(T);
#pragma unroll
    for (int k = 0; k < Raw<T, V>::kWords; ++k) widen_word<T>(r.w[k], &f[k * per]);
  }
}

// acc[v] += a[v] * b[v]: product and sum in fp32, one rounding.  16-bit pairs
// go into the mixed-precision FMA as they lie, without widening.
template <typename T, int V>
__device__ __forceinline__ void fma_raw(const Raw<T, V>& a, const Raw<T, V>& b, float (&acc)[V]) {
  if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) fma_mixed_pair<T>(a.w[k], b.w[k], acc[2 * k], acc[2 * k + 1]);
  } else {
    float x[V], y[V];
    widen<T, V>(a, x);
    widen<T, V>(b, y);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(x[v], y[v], acc[v]);
  }
}

// Two values rounded to nearest even into one word (low half = first).
template <typename T>
__device__ __forceinline__ uint32_t round_pair(float a, float b);
template <>
__device__ __forceinline__ uint32_t round_pair<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t round_pair<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Round to nearest even into the storage type.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> narrow(const float (&f)[V]) {
  Raw<T, V> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < V; ++k) r.w[k] = __float_as_uint(f[k]);
  } else if constexpr (V == 1) {
    const T t = Elem<T>::from_f32(f[0]);
    r.w[0] = *reinterpret_cast<const uint16_t*>(&t);
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) r.w[k] = round_pair<T>(f[2 * k], f[2 * k + 1]);
  }
  return r;
}

// Pairs of fp32 values and their packed arithmetic: one instruction for two
// results, each rounded as its own.
typedef unsigned long long F2;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float lo(F2 p) {
  float a;
  asm("mov.b64 {%0, _}, %1;" : "=f"(a) : "l"(p));
  return a;
}
__device__ __forceinline__ float hi(F2 p) {
  float b;
  asm("mov.b64 {_, %0}, %1;" : "=f"(b) : "l"(p));
  return b;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Tokens in sequence b: lens[b] clamped to 0 ... T, or T.
__device__ __forceinline__ int64_t seq_len(const int32_t* lens, int64_t b, int64_t T) {
  if (lens == nullptr) return T;
  const int64_t n = lens[b];
  return n < 0 ? 0 : n > T ? T : n;
}

// Sum of column `col` of ws [parts][n] by a block of 32 columns x kSumRows
// rows of threads (threadIdx.x = column, threadIdx.y = row): each row adds
// every kSumRows-th part in order, then row 0 adds the rows in order.  The
// order depends on the sizes only.  Returns the sum in row 0.
constexpr int kSumRows = 16;
__device__ __forceinline__ float column_sum(const float* ws, int64_t parts, int64_t n, int64_t col) {
  __shared__ float part[kSumRows][33];
  float s = 0.f;
  if (col < n)
    for (int64_t p = threadIdx.y; p < parts; p += kSumRows) s += ws[p * n + col];
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0)
    for (int r = 1; r < kSumRows; ++r) s += part[r][threadIdx.x];
  return s;
}

}  // namespace gconv
