// Matrices to 8-bit floating point with a scale for each block (gconv_quantize_f8), and the
// residual + root-mean-square norm with such an output (gconv_rms_norm_f8).
//
// For a block with largest magnitude m (at least 2^-110): scale = m / top, f = top / m, and a value's
// number is the one of the format nearest to v f.  That product is not rounded to fp32 first: half of
// the exact ties, of which 16-bit values are full, would go the wrong way.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "plan_cache.h"
#include "seq_vec.cuh"
#include "ssm.h"

namespace gconv {
namespace {

constexpr int kBlk = GCONV_F8_BLOCK;
constexpr float kLeast = 0x1p-110f;

// Two values' codes, the first in the low byte.  v f is cut to 24 bits with what was cut
// kept as the last bit, so that the conversion's rounding is the only one.
__device__ __forceinline__ F2 mul2_rz(F2 a, F2 b) {
  F2 r;
  asm("mul.rz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sticky(float p, float rest) {
  return __uint_as_float(__float_as_uint(p) | (rest != 0.f ? 1u : 0u));
}
template <bool E5>
__device__ __forceinline__ uint32_t codes2(float v0, float v1, float f) {
  const F2 v = f2(v0, v1), p = mul2_rz(v, f2(f, f)), rest = fma2(v, f2(-f, -f), p);
  const float s0 = sticky(lo(p), lo(rest)), s1 = sticky(hi(p), hi(rest));
  uint16_t r;
  if constexpr (E5)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(s1), "f"(s0));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(s1), "f"(s0));
  return r;
}
template <bool E5>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float f) {
  return codes2<E5>(a, b, f) | codes2<E5>(c, d, f) << 16;
}

// A block's two factors, from its largest magnitude as bits (NaN above infinity): no finite one gives f 0 and a
// scale of NaN, and q has to be 0 for all of it.
struct Factor {
  float scale, f;
  bool bad;
};
template <bool E5>
__device__ __forceinline__ Factor factor_of(uint32_t mx) {
  constexpr float top = E5 ? 57344.f : 448.f;
  const float m = fmaxf(__uint_as_float(mx), kLeast);
  const bool bad = mx >= 0x7f800000u;
  return {bad ? __int_as_float(0x7fffffff) : __fdiv_rn(m, top), bad ? 0.f : __fdiv_rn(top, m), bad};
}
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// Largest magnitudes of words as they lie in memory (two 16-bit values a word are taken at once; as whole
// numbers, in which a NaN is above infinity), and then as the bits of an fp32 number.
template <typename T>
__device__ __forceinline__ uint32_t word_max(uint32_t m, uint32_t w) {
  if constexpr (sizeof(T) == 4)
    return max(m, w & 0x7fffffffu);
  else
    return __vmaxu2(m, w & 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ uint32_t half_bits(uint32_t h) {  // of the 16-bit value h, or the 32-bit one
  if constexpr (sizeof(T) == 4)
    return h;
  else if constexpr (std::is_same<T, __nv_bfloat16>::value)
    return h << 16;
  else
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
}
template <typename T>
__device__ __forceinline__ uint32_t max_bits(uint32_t m) {
  return half_bits<T>(sizeof(T) == 4 ? m : max(m & 0xffffu, m >> 16));
}
// Maxima over LANES neighbouring lanes of NV <= LANES values each, as a transposing butterfly: afterwards the lane
// whose place among them is l has that of value l / (LANES / NV).
template <int NV, int LANES>
__device__ __forceinline__ uint32_t lane_max(uint32_t (&v)[NV], int place) {
  int have = NV;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    if (have > 1) {
      const bool up = (place & o) != 0;
      have >>= 1;
#pragma unroll
      for (int k = 0; k < NV / 2; ++k)
        if (k < have) {
          const uint32_t keep = up ? v[k + have] : v[k], send = up ? v[k] : v[k + have];
          v[k] = max(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    } else {
      v[0] = max(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  return v[0];
}

// V codes at q, `left` of which are the row's.
template <int V>
__device__ __forceinline__ void st_codes(uint8_t* q, const uint32_t (&w)[V / 4], int left) {
  if (left >= V) {
    if constexpr (V == 16)
      *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (V == 8)
      *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(q) = w[0];
    return;
  }
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < left) q[e] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
}

// ---------------------------------------------------------------------------
// One block of 256 threads for each 128 x 128 tile of x: warp w has rows 16 w ..., 16 bytes of
// a row a lane, all of its loads in flight at once; a row's factor is computed by one lane and handed
// out.  Rows that vectors do not fit come through shared memory, word by word or element by element.
// For the transposed output the tile is left in shared memory, and a thread takes 16 rows of one
// word's columns: 16 codes, one store.
// 16-bit input is bound by the integer and conversion pipe (76% busy) and issue (71%) more than by memory: some 10
// instructions a value, of which the rounding takes 4.  fp32 has half as many values in the same time, so that something
// else holds it; what has not been measured.  The transposed codes are rounded anew from the tile, for blocks of 128 x
// 128, too.  16384 x 4096 bf16 to e4m3, 1 x 128: 37.5 us, 5.4 TB/s (45 with the maxima and
// the rounding one value at a time); both directions 8192 x 2048 f16 16.5, 8191 x 2050 (by words) 22, 8192 x 8192 bf16
// in 128 x 128 blocks 37.7, the transposed matrix besides 61; fp32 16384 x 2048 35.5; by elements 16384 x 2047 bf16 27.1.
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256, kQWarps = kQThreads / 32, kQRows = kBlk / kQWarps;
enum RowReads { kByVectors, kByWords, kByElements };

template <typename T, bool E5>
__global__ void __launch_bounds__(kQThreads) quant_f8_kernel(QuantF8Args a, RowReads by) {
  constexpr int V = 16 / sizeof(T);
  constexpr int LPR = kBlk / V;        // lanes of a row
  constexpr int RPI = 32 / LPR;        // rows of a warp's load
  constexpr int SETS = kQRows / RPI;
  constexpr int CW = 4 / sizeof(T);    // columns of a word
  constexpr int WORDS = kBlk / CW;     // of a row
  constexpr int CHUNKS = kBlk / 16;    // of 16 rows
  constexpr int MINE = WORDS * CHUNKS / kQThreads;
  extern __shared__ __align__(16) unsigned char smem[];
  T* const tile = reinterpret_cast<T*>(smem);  // [128][128], where it is needed
  __shared__ uint32_t part[CHUNKS][WORDS];
  __shared__ float col_f[kBlk];
  __shared__ uint32_t all;
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t nb = (a.D + kBlk - 1) / kBlk, rb = blockIdx.x / nb, kb = blockIdx.x - rb * nb;
  const int64_t r0 = rb * kBlk, c0 = kb * kBlk;
  const int rows = a.rows - r0 < kBlk ? (int)(a.rows - r0) : kBlk, cols = a.D - c0 < kBlk ? (int)(a.D - c0) : kBlk;
  const bool square = a.block_rows != 1;
  grid_dependency_wait();
  const T* x = static_cast<const T*>(a.x) + r0 * a.sx + c0;
  if (threadIdx.x == 0) all = 0;
  if (by != kByVectors) {
    const int first = warp * kQRows;
    if (by == kByWords) {
#pragma unroll 8
      for (int r = first; r < first + kQRows; ++r)
#pragma unroll
        for (int w = lane; w < WORDS; w += 32)
          reinterpret_cast<uint32_t*>(tile)[r * WORDS + w] =
              r < rows && w * CW < cols ? *reinterpret_cast<const uint32_t*>(x + r * a.sx + w * CW) : 0u;
    } else {
#pragma unroll 8
      for (int r = first; r < first + kQRows; ++r)
#pragma unroll
        for (int c = lane; c < kBlk; c += 32) tile[r * kBlk + c] = r < rows && c < cols ? x[r * a.sx + c] : Elem<T>::from_f32(0.f);
    }
    __syncwarp();
  }
  const int place = lane % LPR, sub = lane / LPR, e0 = place * V;
  Raw<T, V> v[SETS];
#pragma unroll
  for (int k = 0; k < SETS; ++k) {
    const int r = warp * kQRows + k * RPI + sub;
    if (by != kByVectors)
      v[k] = ld_raw<T, V>(tile + r * kBlk + e0);
    else
      v[k] = r < rows && e0 < cols ? ld_raw<T, V>(x + r * a.sx + e0) : zero_raw<T, V>();
  }
  if (by == kByVectors && a.qt)
#pragma unroll
    for (int k = 0; k < SETS; ++k) st_raw<T, V>(tile + (warp * kQRows + k * RPI + sub) * kBlk + e0, v[k]);
  uint32_t mx[SETS];
#pragma unroll
  for (int k = 0; k < SETS; ++k) {
    mx[k] = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) mx[k] = word_max<T>(mx[k], v[k].w[w]);
  }
  Factor mine = {};  // of a row; squares: of the block
  if (square) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < SETS; ++k) m = word_max<T>(m, mx[k]);
    m = __reduce_max_sync(0xffffffffu, max_bits<T>(m));
    __syncthreads();
    if (lane == 0) atomicMax(&all, m);
    __syncthreads();
    mine = factor_of<E5>(all);
    if (threadIdx.x == 0) {
      if (a.q) a.scale[kb * a.ss + rb] = mine.scale;
      if (a.qt) a.scale_t[rb * a.sst + kb] = mine.scale;
    }
  } else if (a.q) {
#pragma unroll
    for (int k = 0; k < SETS; ++k) mx[k] = max_bits<T>(mx[k]);
    mine = factor_of<E5>(lane_max<SETS, LPR>(mx, place));
    constexpr int EACH = LPR / SETS;  // lanes with a row's factor
    const int r = warp * kQRows + place / EACH * RPI + sub;
    if (place % EACH == 0 && r < rows) a.scale[kb * a.ss + r0 + r] = mine.scale;
  }
  if (a.q) {
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
      const int r = warp * kQRows + k * RPI + sub;
      const float f = square ? mine.f : __shfl_sync(0xffffffffu, mine.f, sub * LPR + k * (LPR / SETS));
      float w[V];
      widen<T, V>(v[k], w);
      uint32_t q[V / 4];
#pragma unroll
      for (int e = 0; e < V / 4; ++e) {
        const uint32_t c = codes4<E5>(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3], f);
        q[e] = f == 0.f ? 0u : c;  // no finite largest value
      }
      if (r < rows) st_codes<V>(a.q + (r0 + r) * a.qp + c0 + e0, q, cols - e0);
    }
  }
  if (a.qt == nullptr) return;
  __syncthreads();
  uint32_t raw[MINE][16];
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    const int at = threadIdx.x + k * kQThreads, word = at % WORDS, chunk = at / WORDS;
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      raw[k][r] = reinterpret_cast<const uint32_t*>(tile)[(chunk * 16 + r) * WORDS + word];
      m = word_max<T>(m, raw[k][r]);
    }
    part[chunk][word] = m;
  }
  if (!square) {
    __syncthreads();
    if (threadIdx.x < kBlk) {
      const int c = threadIdx.x;
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < CHUNKS; ++k) m = word_max<T>(m, part[k][c / CW]);
      const Factor f = factor_of<E5>(half_bits<T>(CW == 1 ? m : c & 1 ? m >> 16 : m & 0xffffu));
      col_f[c] = f.f;
      if (c < cols) a.scale_t[rb * a.sst + c0 + c] = f.scale;
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    const int at = threadIdx.x + k * kQThreads, word = at % WORDS, chunk = at / WORDS;
#pragma unroll
    for (int j = 0; j < CW; ++j) {
      const int c = word * CW + j;
      const float f = square ? mine.f : col_f[c];
      uint32_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float two[CW];
          widen_word<T>(raw[k][4 * e + i], two);
          w[i] = two[j];
        }
        const uint32_t codes = codes4<E5>(w[0], w[1], w[2], w[3], f);
        q[e] = f == 0.f ? 0u : codes;
      }
      if (c < cols) st_codes<16>(a.qt + (c0 + c) * a.qtp + r0 + chunk * 16, q, rows - chunk * 16);
    }
  }
}

template <typename T, bool E5>
cudaError_t launch_quant(const QuantF8Args& q, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int V = 16 / sizeof(T);
  constexpr int CW = 4 / sizeof(T);
  const uintptr_t at = reinterpret_cast<uintptr_t>(q.x);
  const RowReads by = q.sx % V == 0 && q.D % V == 0 && at % 16 == 0     ? kByVectors
                      : q.sx % CW == 0 && q.D % CW == 0 && at % 4 == 0 ? kByWords
                                                                       : kByElements;
  const size_t smem = by != kByVectors || q.qt ? kBlk * kBlk * sizeof(T) : 0;
  if (smem > 40 * 1024) {  // 48 KB less what the kernel declares is there without asking
    static SmemAttr attr;
    const cudaError_t e = attr.ensure(quant_f8_kernel<T, E5>, dev.device, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int64_t blocks = (q.rows + kBlk - 1) / kBlk * ((q.D + kBlk - 1) / kBlk);
  return launch_kernel(quant_f8_kernel<T, E5>, dim3((unsigned)blocks), dim3(kQThreads), smem, a, q, by);
}

// ---------------------------------------------------------------------------
// Norm.  q needs no statistics of the row (the row's factor is the same for all of a block and goes into its
// scale), so it is written while the sum of squares is still being taken.  Bound by memory: 16384 x 4096 bf16 71.4 us,
// 97% of the measured copy rate (78 with the rounding one value at a time); 16 x 2048 2.1, the launch and one way
// through the row.  Rows off 16 bytes come by aligned words, four or five a thread and vector, whose lines the
// threads of a warp share: bound by those loads and the joining.  16384 x 4095 bf16 152 us, 8192 x 4095 fp32 76,
// 40000 x 701 bf16 86, 200 x 2047 3.7; with the row in shared memory, element by element, 176, 102, 124 and 5.0.
// That form is left for rows wider than registers (fp32 8192, else 16384 elements).
// ---------------------------------------------------------------------------
// Rows whose squares come near the smallest fp32 numbers: the sum is taken again of h times 2^100.
constexpr float kTiny = 0x1p-110f, kLift = 0x1p100f;
// 1 / sqrt(mean + eps) from the sum as it was and, for a tiny one, of the lifted values.
__device__ __forceinline__ float root_of(const NormF8Args& n, float sum, float lifted_sum, bool lift) {
  if (lift && n.eps < kTiny) {
    const float ms = lifted_sum / (float)n.D + n.eps * kLift * kLift;
    return ms > 0.f ? rsqrtf(ms) * kLift : ms == 0.f ? 0.f : ms;
  }
  const float ms = sum / (float)n.D + n.eps;
  return ms > 0.f ? rsqrtf(ms) : ms == 0.f ? 0.f : ms;  // NaN stays
}
// A block's largest magnitude where the row's sum is not finite: none.
__device__ __forceinline__ uint32_t block_top(uint32_t mx, bool bad) { return bad ? 0x7fffffffu : mx; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float sums[32];
  const int warps = (blockDim.x + 31) / 32, lane = threadIdx.x & 31;
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? sums[lane] : 0.f);
}

// Rows wider than registers: one block for each row, the row's h in shared memory, blocks of 128 by warps.
template <typename T, bool E5>
__global__ void __launch_bounds__(256) norm_f8_any_kernel(NormF8Args n) {
  extern __shared__ __align__(16) unsigned char smem[];
  T* hs = reinterpret_cast<T*>(smem);
  allow_dependent_launch();
  grid_dependency_wait();
  const int64_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* x = static_cast<const T*>(n.x) + row * n.sx;
  const T* res = n.res ? static_cast<const T*>(n.res) + row * n.sr : nullptr;
  const T* w = static_cast<const T*>(n.w);
  T* ro = n.res_out ? static_cast<T*>(n.res_out) + row * n.sr : nullptr;
  float sum = 0.f;
  constexpr int kAtOnce = 8;  // elements a thread asks for together
  for (int k0 = threadIdx.x; k0 < n.D; k0 += kAtOnce * 256) {
    T hx[kAtOnce], hr[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const bool in = k0 + 256 * j < n.D;
      hx[j] = in ? x[k0 + 256 * j] : Elem<T>::from_f32(0.f);
      hr[j] = in && res ? res[k0 + 256 * j] : Elem<T>::from_f32(0.f);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int k = k0 + 256 * j;
      if (k >= n.D) break;
      T h = hx[j];
      if (res) h = Elem<T>::from_f32(Elem<T>::to_f32(h) + Elem<T>::to_f32(hr[j]));
      if (ro) ro[k] = h;
      hs[k] = h;
      const float f = Elem<T>::to_f32(h);
      sum = fmaf(f, f, sum);
    }
  }
  sum = block_sum(sum);
  const bool lift = !std::is_same<T, __half>::value && sum < kTiny, bad = !(sum < INFINITY);
  float lifted = 0.f;
  if (lift) {  // the whole block
    for (int k = threadIdx.x; k < n.D; k += blockDim.x) {
      const float f = Elem<T>::to_f32(hs[k]) * kLift;
      lifted = fmaf(f, f, lifted);
    }
    lifted = block_sum(lifted);
  }
  const float root = root_of(n, sum, lifted, lift);
  const int blocks = (n.D + kBlk - 1) / kBlk;
#pragma unroll 2
  for (int kb = warp; kb < blocks; kb += 8) {
    float u[4];
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = kb * kBlk + 32 * j + lane;
      u[j] = k < n.D ? Elem<T>::to_f32(hs[k]) * (w ? Elem<T>::to_f32(w[k]) : 1.f) : 0.f;
      mx = max(mx, mag(u[j]));
      if (n.y && k < n.D) static_cast<T*>(n.y)[row * n.sy + k] = Elem<T>::from_f32(u[j] * root);
    }
    if (n.q == nullptr) continue;
    const Factor f = factor_of<E5>(block_top(__reduce_max_sync(0xffffffffu, mx), bad));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = kb * kBlk + 32 * j + lane;
      if (k < n.D) n.q[row * n.qp + k] = f.bad ? (uint8_t)0 : (uint8_t)codes2<E5>(u[j], 0.f, f.f);
    }
    if (lane == 0) n.scale[(int64_t)kb * n.rows + row] = f.scale * root;
  }
}

// 16 bytes' elements from p on, `left` of them the row's and the rest zeros, from and to any address: by the aligned
// words that hold any of them, joined by shifts.  The first and the last word may hold a half of what lies beside them:
// a matrix's first and last vectors (end_vector), beside which nothing may lie, come by elements.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> ld_words(const T* p, int left, bool end) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint32_t* from = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
  Raw<T, V> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) r.w[k] = k < left ? from[k] : 0u;
  } else {
    if (end) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint16_t* const two = reinterpret_cast<const uint16_t*>(p) + 2 * k;
        r.w[k] = (2 * k < left ? two[0] : 0u) | (2 * k + 1 < left ? (uint32_t)two[1] << 16 : 0u);
      }
      return r;
    }
    const int off = (int)(at & 2) / 2, have = left < V ? left : V;
    uint32_t v[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) v[k] = left > 0 && 2 * k < have + off ? from[k] : 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t two = __funnelshift_r(v[k], v[k + 1], 16 * off);
      r.w[k] = 2 * k + 1 < left ? two : 2 * k < left ? two & 0xffffu : 0u;
    }
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void st_words(T* p, const Raw<T, V>& r, int left) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) reinterpret_cast<uint32_t*>(p)[k] = r.w[k];
  } else {
    uint16_t* const to = reinterpret_cast<uint16_t*>(p);
    if (left < V) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < left) to[e] = (uint16_t)(r.w[e / 2] >> (16 * (e & 1)));
    } else if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) reinterpret_cast<uint32_t*>(to)[k] = r.w[k];
    } else {
      to[0] = (uint16_t)r.w[0];
#pragma unroll
      for (int k = 0; k < 3; ++k) reinterpret_cast<uint32_t*>(to + 1)[k] = __funnelshift_r(r.w[k], r.w[k + 1], 16);
      to[V - 1] = (uint16_t)(r.w[3] >> 16);
    }
  }
}

// A thread keeps NV vectors of 16 bytes of its block's row in registers, so the row is
// read once.  A block of 128 is 16 lanes' vectors (fp32: 32).
// WARP: a row is a warp's, kRowWarps of them in a block.  WORDS: rows of any width, stride and alignment.
constexpr int kRowWarps = 4;
template <typename T, bool E5, int NV, bool WARP, bool WORDS>
__global__ void __launch_bounds__(512) norm_f8_vec_kernel(NormF8Args n) {
  constexpr int V = 16 / sizeof(T), LPB = kBlk / V;
  allow_dependent_launch();
  const int threads = WARP ? 32 : (int)blockDim.x, self = WARP ? (int)threadIdx.x & 31 : (int)threadIdx.x;
  const int64_t row = WARP ? blockIdx.x * (int64_t)kRowWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (WARP && row >= n.rows) return;
  const T* x = static_cast<const T*>(n.x) + row * n.sx;
  const T* res = n.res ? static_cast<const T*>(n.res) + row * n.sr : nullptr;
  const T* w = static_cast<const T*>(n.w);
  T* ro = n.res_out ? static_cast<T*>(n.res_out) + row * n.sr : nullptr;
  auto put = [](T* p, const Raw<T, V>& v, int left) {
    if constexpr (WORDS)
      st_words<T, V>(p, v, left);
    else
      st_raw<T, V>(p, v);
  };
  grid_dependency_wait();
  Raw<T, V> h[NV], r[NV], g[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = (k * threads + self) * V;
    const bool in = e < n.D;
    auto from = [&](const T* p, int64_t r, int64_t rows) -> Raw<T, V> {  // of row r of `rows`
      if constexpr (WORDS)
        return ld_words<T, V>(p + e, n.D - e, end_vector(r, e, rows, n.D, V));
      else
        return ld_raw<T, V>(p + e);
    };
    h[k] = in ? from(x, row, n.rows) : zero_raw<T, V>();
    r[k] = in && res ? from(res, row, n.rows) : zero_raw<T, V>();
    g[k] = in && w ? from(w, 0, 1) : zero_raw<T, V>();
  }
  float sum = 0.f;
  uint32_t mx[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = (k * threads + self) * V;
    float f[V], gf[V];
    widen<T, V>(h[k], f);
    if (res) {
      float o[V];
      widen<T, V>(r[k], o);
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] += o[v];
      h[k] = narrow<T, V>(f);
      widen<T, V>(h[k], f);
    }
    if (ro && e < n.D) put(ro + e, h[k], n.D - e);
    widen<T, V>(g[k], gf);
    mx[k] = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      sum = fmaf(f[v], f[v], sum);
      mx[k] = max(mx[k], mag(w ? f[v] * gf[v] : f[v]));
    }
  }
  const uint32_t top = lane_max<NV, LPB>(mx, self % LPB);
  auto total = [&](float v) { return WARP ? warp_sum(v) : block_sum(v); };
  sum = total(sum);
  const bool lift = !std::is_same<T, __half>::value && sum < kTiny, bad = !(sum < INFINITY);
  float lifted = 0.f;
  if (lift) {  // the whole warp or block
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float f[V];
      widen<T, V>(h[k], f);
#pragma unroll
      for (int v = 0; v < V; ++v) lifted = fmaf(f[v] * kLift, f[v] * kLift, lifted);
    }
    lifted = total(lifted);
  }
  const float root = root_of(n, sum, lifted, lift);
  // a lane has the factor of one of its group's NV blocks
  const Factor mine = factor_of<E5>(block_top(top, bad));
  constexpr int EACH = LPB / NV;
  if (n.q && self % EACH == 0) {
    const int e = (self % LPB / EACH * threads + self / LPB * LPB) * V;
    if (e < n.D) n.scale[(int64_t)(e / kBlk) * n.rows + row] = mine.scale * root;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = (k * threads + self) * V;
    const float to = __shfl_sync(0xffffffffu, mine.f, (self & 31) / LPB * LPB + k * EACH);
    if (e >= n.D) continue;
    float f[V], gf[V];
    widen<T, V>(h[k], f);
    widen<T, V>(g[k], gf);
    if (w) {
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] *= gf[v];
    }
    if (n.q) {
      uint32_t q[V / 4];
#pragma unroll
      for (int v = 0; v < V / 4; ++v) {
        const uint32_t c = codes4<E5>(f[4 * v], f[4 * v + 1], f[4 * v + 2], f[4 * v + 3], to);
        q[v] = to == 0.f ? 0u : c;  // no finite largest value
      }
      st_codes<V>(n.q + row * n.qp + e, q, WORDS ? n.D - e : V);
    }
    if (n.y) {
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] *= root;
      put(static_cast<T*>(n.y) + row * n.sy + e, narrow<T, V>(f), n.D - e);
    }
  }
}

bool norm_vectors(const NormF8Args& n, int V) {
  for (int64_t s : {n.sx, n.res ? n.sr : 0, n.res_out ? n.sr : 0, n.y ? n.sy : 0, (int64_t)n.D})
    if (s % V != 0) return false;
  for (const void* p : {n.x, n.res, n.w, (const void*)n.res_out, (const void*)n.y})
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return true;
}

template <typename T, bool E5, bool WORDS>
cudaError_t launch_rows(const NormF8Args& n, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int V = 16 / sizeof(T);
  // few rows: one vector a thread; short rows a warp each; else four vectors a thread
  const int vectors = (n.D + V - 1) / V;
  const dim3 grid((unsigned)n.rows), warps((unsigned)((n.rows + kRowWarps - 1) / kRowWarps));
  auto threads = [&](int nv) { return ((vectors + nv - 1) / nv + 31) / 32 * 32; };
  if (threads(1) <= 512 && n.rows < 4 * dev.num_sms)
    return launch_kernel(norm_f8_vec_kernel<T, E5, 1, false, WORDS>, grid, dim3(threads(1)), 0, a, n);
  if (vectors <= 32) return launch_kernel(norm_f8_vec_kernel<T, E5, 1, true, WORDS>, warps, dim3(32 * kRowWarps), 0, a, n);
  if (vectors <= 64) return launch_kernel(norm_f8_vec_kernel<T, E5, 2, true, WORDS>, warps, dim3(32 * kRowWarps), 0, a, n);
  if (vectors <= 128) return launch_kernel(norm_f8_vec_kernel<T, E5, 4, true, WORDS>, warps, dim3(32 * kRowWarps), 0, a, n);
  return launch_kernel(norm_f8_vec_kernel<T, E5, 4, false, WORDS>, grid, dim3(threads(4)), 0, a, n);
}

template <typename T, bool E5>
cudaError_t launch_norm(const NormF8Args& n, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int V = 16 / sizeof(T);
  if (n.D <= 512 * 4 * V)
    return norm_vectors(n, V) ? launch_rows<T, E5, false>(n, a, dev) : launch_rows<T, E5, true>(n, a, dev);
  const size_t smem = (size_t)n.D * sizeof(T);
  if (smem > 47 * 1024) {  // 48 KB less the reductions' few bytes is there without asking
    static SmemAttr attr;
    const cudaError_t e = attr.ensure(norm_f8_any_kernel<T, E5>, dev.device, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(norm_f8_any_kernel<T, E5>, dim3((unsigned)n.rows), dim3(256), smem, a, n);
}

}  // namespace

cudaError_t quant_f8_launch(const QuantF8Args& q, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (a.dt) {
    case kF32: return q.e5 ? launch_quant<float, true>(q, a, dev) : launch_quant<float, false>(q, a, dev);
    case kF16: return q.e5 ? launch_quant<__half, true>(q, a, dev) : launch_quant<__half, false>(q, a, dev);
    default: return q.e5 ? launch_quant<__nv_bfloat16, true>(q, a, dev) : launch_quant<__nv_bfloat16, false>(q, a, dev);
  }
}

cudaError_t norm_f8_launch(const NormF8Args& n, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (a.dt) {
    case kF32: return n.e5 ? launch_norm<float, true>(n, a, dev) : launch_norm<float, false>(n, a, dev);
    case kF16: return n.e5 ? launch_norm<__half, true>(n, a, dev) : launch_norm<__half, false>(n, a, dev);
    default: return n.e5 ? launch_norm<__nv_bfloat16, true>(n, a, dev) : launch_norm<__nv_bfloat16, false>(n, a, dev);
  }
}

}  // namespace gconv
