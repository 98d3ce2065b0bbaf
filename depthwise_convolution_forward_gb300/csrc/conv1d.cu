// Causal depthwise convolution along a sequence (gconv_causal_conv1d_*).
//
//   u_t = bias + sum_j w_j e_{t-(K-1)+j},  y_t = act(u_t)
//
// with e the sequence and, before it, the K - 1 carried rows.
#include <initializer_list>

#include "seq.h"
#include "seq_vec.cuh"

namespace gconv {
namespace {

constexpr int kMaxK = GCONV_CONV1D_MAX_K;

__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// Row t of e for V channels from d, as it lies in memory: the sequence, the
// carried rows before it, zeros before those or past its end n.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> ext_raw(const ConvSeqArgs& c, const T* x, const T* state, int K, int64_t t,
                                             int64_t n) {
  if (t >= 0) return t < n ? ld_raw<T, V>(x + t * c.sx.t) : zero_raw<T, V>();
  return state != nullptr && t >= 1 - K ? ld_raw<T, V>(state + (t + K - 1) * (int64_t)c.D) : zero_raw<T, V>();
}

// The filter's taps: KT where the kernel is made for that many.
template <int KT>
__device__ __forceinline__ int taps_of(const ConvSeqArgs& c) {
  return KT <= 4 ? KT : c.K;
}

// Weights of V channels from d for KT taps, [tap][channel] as raw values.  The V K
// weights lie together, so four channels of a filter of KT taps come as KT
// vectors; a filter of K < KT taps is placed at the end, and its first KT - K
// taps are skipped.
template <typename T, int V, int KT>
__device__ __forceinline__ void load_taps(const ConvSeqArgs& c, int d, Raw<T, V> (&w)[KT]) {
  const int K = taps_of<KT>(c);
  const T* p = static_cast<const T*>(c.w) + (int64_t)d * K;
  if constexpr (KT <= 4 && V == 4) {
    Raw<T, 4> row[KT];  // elements 4 k ... 4 k + 3 of the V K
#pragma unroll
    for (int k = 0; k < KT; ++k) row[k] = ld_raw<T, 4>(p + 4 * k);
    auto at = [&](int e) {  // element e, as bits
      if constexpr (sizeof(T) == 4)
        return row[e / 4].w[e % 4];
      else
        return e % 2 ? row[e / 4].w[e % 4 / 2] >> 16 : row[e / 4].w[e % 4 / 2] & 0xffffu;
    };
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int v = 0; v < 4; ++v) w[j].w[v] = at(v * KT + j);
      } else {
        w[j].w[0] = at(j) | at(KT + j) << 16;
        w[j].w[1] = at(2 * KT + j) | at(3 * KT + j) << 16;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      const int k = j - (KT - K);
      uint32_t e[V];
#pragma unroll
      for (int v = 0; v < V; ++v) e[v] = k >= 0 ? ld_raw<T, 1>(p + v * K + k).w[0] : 0u;
      if constexpr (sizeof(T) == 4 || V == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) w[j].w[v] = e[v];
      } else {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) w[j].w[v] = e[2 * v] | e[2 * v + 1] << 16;
      }
    }
  }
}

// Sequence and tile of the flat index q = b * tiles + tile.
__device__ __forceinline__ void split_index(int64_t q, int64_t tiles, int64_t* b, int64_t* tile) {
  if (tiles == 1) {
    *b = q, *tile = 0;
  } else if (q < (int64_t)1 << 31 && tiles < (int64_t)1 << 31) {
    const uint32_t u = (uint32_t)q / (uint32_t)tiles;
    *b = u, *tile = (uint32_t)q - u * (uint32_t)tiles;
  } else {
    *b = q / tiles, *tile = q - *b * tiles;
  }
}

// Forward.  A thread owns V channels and nb batches of kRows tokens of one
// sequence; a batch's rows are loaded together, so that enough of them are
// in flight, and the K - 1 rows before them stay in registers.  The thread of
// a sequence's first tokens, the only one that reads the state, also moves it:
// it reads what went in before it writes what comes out, so the two may be the
// same.
constexpr int kFwdY = 4;  // threads of a block along the flat (sequence, tile) index
template <typename T, int V, int KT, int kRows>
__global__ void __launch_bounds__(32 * kFwdY, sizeof(T) == 2 && KT <= 4 ? 8 : 1)
conv1d_fwd_kernel(ConvSeqArgs c, int nb, int64_t tiles, int dblocks) {
  const int K = taps_of<KT>(c);
  allow_dependent_launch();
  const int64_t qb = blockIdx.x / (uint32_t)dblocks;
  const int d = ((int)(blockIdx.x - (uint32_t)qb * (uint32_t)dblocks) * 32 + threadIdx.x) * V;
  int64_t b, tile;
  split_index(qb * kFwdY + threadIdx.y, tiles, &b, &tile);
  if (d >= c.D || b >= c.B) return;
  const int64_t t0 = tile * nb * kRows;
  const T* x = static_cast<const T*>(c.x) + b * c.sx.b + d;
  T* y = static_cast<T*>(c.y) + b * c.sy.b + t0 * c.sy.t + d;
  const T* state = c.state_in ? static_cast<const T*>(c.state_in) + b * (K - 1) * (int64_t)c.D + d : nullptr;
  grid_dependency_wait();
  const int64_t n = seq_len(c.lens, b, c.T);
  // tokens of this thread that exist, and that lie inside the sequence
  const int span = nb * kRows;
  const int rows = c.T - t0 < span ? (int)(c.T - t0) : span, live = n - t0 < rows ? (n > t0 ? (int)(n - t0) : 0) : rows;
  Raw<T, V> raw[kRows], win[KT], w[KT];
  const T* from = x + t0 * c.sx.t;
  auto load = [&](int r) {  // the batch from row r
    if (r + kRows <= live) {
#pragma unroll
      for (int k = 0; k < kRows; ++k) raw[k] = ld_raw<T, V>(from + (int64_t)k * c.sx.t);
    } else {
#pragma unroll
      for (int k = 0; k < kRows; ++k) raw[k] = r + k < live ? ld_raw<T, V>(from + (int64_t)k * c.sx.t) : zero_raw<T, V>();
    }
    from += (int64_t)kRows * c.sx.t;
  };
  load(0);
#pragma unroll
  for (int j = 0; j < KT - 1; ++j) win[j] = ext_raw<T, V>(c, x, state, K, t0 - (KT - 1) + j, n);
  float bias[V];
  load_taps<T, V, KT>(c, d, w);
  widen<T, V>(c.bias ? ld_raw<T, V>(static_cast<const T*>(c.bias) + d) : zero_raw<T, V>(), bias);
  if (KT > 1 && c.state_out && tile == 0) {
    // Rows n - (K - 1) ... n - 1 of e, all read before the first is written: the
    // state that comes out may be the one that went in.
    T* out = static_cast<T*>(c.state_out) + b * (K - 1) * (int64_t)c.D + d;
    Raw<T, V> last[KT];
#pragma unroll
    for (int j = 0; j < KT - 1; ++j)
      if (j >= KT - K) last[j] = ext_raw<T, V>(c, x, state, K, n - (KT - 1) + j, n);
#pragma unroll
    for (int j = 0; j < KT - 1; ++j)
      if (j >= KT - K) st_raw<T, V>(out + (int64_t)(j - (KT - K)) * c.D, last[j]);
  }
  for (int r = 0; r < rows; r += kRows) {
    Raw<T, V> cur[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) cur[k] = raw[k];
    load(r + kRows);  // on its way while this batch is computed; nothing past the last
    const bool whole = r + kRows <= live;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      win[KT - 1] = cur[k];
      float u[V];
#pragma unroll
      for (int v = 0; v < V; ++v) u[v] = bias[v];
#pragma unroll
      for (int j = 0; j < KT; ++j)
        if (j >= KT - K) fma_raw<T, V>(win[j], w[j], u);
      if (c.act) {
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] *= sigmoid(u[v]);
      }
      if (whole || r + k < rows) st_raw<T, V>(y, whole || r + k < live ? narrow<T, V>(u) : zero_raw<T, V>());
      y += c.sy.t;
#pragma unroll
      for (int j = 0; j < KT - 1; ++j) win[j] = win[j + 1];
    }
  }
}

// Backward.  A thread owns V channels and kSteps tokens; it walks them and the
// K - 1 after them, which its last rows of dx need, keeping the last K rows of e
// and of du.  Once du_t is known, row p = t - (K - 1) is complete:
//   de_p = sum_j w_j du_{p + K - 1 - j},   dw_j += e_p du_{p + K - 1 - j}
// so each row of e is widened once, when it is the oldest.  The sums for dw and
// dbias are added over the block's kBwdY threads along time in shared memory and
// leave as one row of partial sums [K + 1][D] for each block of tokens.
constexpr int kSteps = 32;
constexpr int kBwdY = 4;
constexpr int kBwdTile = kSteps * kBwdY;
template <typename T, int V, int KT>
__global__ void __launch_bounds__(32 * kBwdY, KT <= 4 ? 3 : 1)
conv1d_bwd_kernel(ConvSeqArgs c, int64_t tiles, int dblocks) {
  __shared__ float part[kBwdY][32][V + 1];
  const int K = taps_of<KT>(c);
  allow_dependent_launch();
  const int64_t q = blockIdx.x / (uint32_t)dblocks;
  const int d = ((int)(blockIdx.x - (uint32_t)q * (uint32_t)dblocks) * 32 + threadIdx.x) * V;
  int64_t b, tile;
  split_index(q, tiles, &b, &tile);
  const int64_t t0 = tile * kBwdTile + threadIdx.y * kSteps;
  const bool mine = d < c.D;
  grid_dependency_wait();
  const int64_t n = seq_len(c.lens, b, c.T);
  float dw[KT][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int j = 0; j < KT; ++j) dw[j][v] = 0.f;
  }
  if (mine && t0 < c.T && t0 >= n && t0 > 0) {
    // past the sequence's end
    const int own = c.T - t0 < kSteps ? (int)(c.T - t0) : kSteps;
    T* pd = static_cast<T*>(c.dx) + b * c.sx.b + t0 * c.sx.t + d;
    for (int r = 0; r < own; ++r, pd += c.sx.t) st_raw<T, V>(pd, zero_raw<T, V>());
  } else if (mine && t0 < c.T) {
    const int64_t K1 = K - 1;
    const T* x = static_cast<const T*>(c.x) + b * c.sx.b + d;
    const T* dy = static_cast<const T*>(c.dy) + b * c.sy.b + d;
    T* dx = static_cast<T*>(c.dx) + b * c.sx.b + d;
    const T* state = c.state_in ? static_cast<const T*>(c.state_in) + b * K1 * c.D + d : nullptr;
    const T* dso = c.dstate_out ? static_cast<const T*>(c.dstate_out) + b * K1 * c.D + d : nullptr;
    T* dsi = c.dstate_in ? static_cast<T*>(c.dstate_in) + b * K1 * c.D + d : nullptr;
    Raw<T, V> wr[KT], win[KT];  // as they lie in memory: fewer registers
    float wf[KT][V], bias[V], du[KT][V];
    load_taps<T, V, KT>(c, d, wr);
#pragma unroll
    for (int j = 0; j < KT; ++j) widen<T, V>(wr[j], wf[j]);
    widen<T, V>(c.bias ? ld_raw<T, V>(static_cast<const T*>(c.bias) + d) : zero_raw<T, V>(), bias);
#pragma unroll
    for (int j = 0; j < KT - 1; ++j) {
      win[j] = ext_raw<T, V>(c, x, state, K, t0 - (KT - 1) + j, n);
#pragma unroll
      for (int v = 0; v < V; ++v) du[j][v] = 0.f;
    }
    // counted from t0: tokens of this thread, tokens to walk, tokens inside the
    // sequence, and the first row p that is this thread's (the first thread of a
    // sequence also has the carried rows)
    const int own = c.T - t0 < kSteps ? (int)(c.T - t0) : kSteps, walk = own + K - 1;
    const int live = n - t0 < walk ? (n > t0 ? (int)(n - t0) : 0) : walk;
    const int p0 = t0 == 0 ? 1 - K : 0;
    const bool ends = dso != nullptr && n - (K - 1) < t0 + own && n > t0 + p0;  // some of its rows leave with the state
    constexpr int kBatch = 4;
    const T *px = x + t0 * c.sx.t, *pg = dy + t0 * c.sy.t;
    T* pd = dx + (t0 - (K - 1)) * c.sx.t;
    Raw<T, V> nx[kBatch], ng[kBatch];
    auto load = [&](int r) {
      const bool all = r + kBatch <= live;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        nx[k] = all || r + k < live ? ld_raw<T, V>(px) : zero_raw<T, V>();
        ng[k] = all || r + k < live ? ld_raw<T, V>(pg) : zero_raw<T, V>();
        px += c.sx.t, pg += c.sy.t;
      }
    };
    load(0);
    for (int r = 0; r < walk; r += kBatch) {
      Raw<T, V> rx[kBatch], rg[kBatch];
      const bool whole = r + kBatch <= live;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) rx[k] = nx[k], rg[k] = ng[k];
      load(r + kBatch);  // on its way while this batch is computed
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        win[KT - 1] = rx[k];
        widen<T, V>(rg[k], du[KT - 1]);  // past the end of the sequence dy was read as 0
        if (c.act) {
          float u[V];
#pragma unroll
          for (int v = 0; v < V; ++v) u[v] = bias[v];
#pragma unroll
          for (int j = 0; j < KT; ++j)
            if (j >= KT - K) fma_raw<T, V>(win[j], wr[j], u);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float g = sigmoid(u[v]);
            du[KT - 1][v] *= g * fmaf(u[v], 1.f - g, 1.f);
          }
          if (!whole && r + k >= live) {
#pragma unroll
            for (int v = 0; v < V; ++v) du[KT - 1][v] = 0.f;
          }
        }
        const int p = r + k - (K - 1);
        if (p >= p0 && r + k < walk) {
          float de[V], e[V];
          const int oldest = KT - K;  // of the windows' rows
#pragma unroll
          for (int m = 0; m < KT; ++m)
            if (m == oldest) {
              widen<T, V>(win[m], e);
#pragma unroll
              for (int v = 0; v < V; ++v) db[v] += du[m][v], de[v] = 0.f;
            }
          // tap j meets du_{p + K - 1 - j}, row KT - 1 - (j - oldest) of du
#pragma unroll
          for (int j = 0; j < KT; ++j)
            if (j >= KT - K) {
#pragma unroll
              for (int m = 0; m < KT; ++m)
                if (m == KT - 1 - (j - oldest))
#pragma unroll
                  for (int v = 0; v < V; ++v) {
                    de[v] = fmaf(wf[j][v], du[m][v], de[v]);
                    dw[j][v] = fmaf(e[v], du[m][v], dw[j][v]);
                  }
            }
          if (ends) {
            const int64_t row = t0 + p - (n - (K - 1));
            if (row >= 0 && row < K - 1) {
              float o[V];
              widen<T, V>(ld_raw<T, V>(dso + row * c.D), o);
#pragma unroll
              for (int v = 0; v < V; ++v) de[v] += o[v];
            }
          }
          if (p >= 0)
            st_raw<T, V>(pd, narrow<T, V>(de));
          else if (dsi != nullptr)
            st_raw<T, V>(dsi + (int64_t)(p + K - 1) * c.D, narrow<T, V>(de));
        }
        pd += c.sx.t;
#pragma unroll
        for (int j = 0; j < KT - 1; ++j) {
          win[j] = win[j + 1];
#pragma unroll
          for (int v = 0; v < V; ++v) du[j][v] = du[j + 1][v];
        }
      }
    }
    // Past the end dx is 0, whatever the weights: one that is not finite has made
    // NaN of the zeros there.
    pd = dx + (t0 + live) * c.sx.t;
    for (int r = live; r < own; ++r, pd += c.sx.t) st_raw<T, V>(pd, zero_raw<T, V>());
  }
  // [K + 1][D] sums of the block: kBwdY threads of each channel, in order
  float* ws = c.ws + q * (K + 1) * (int64_t)c.D;
#pragma unroll
  for (int j = 0; j <= KT; ++j) {
    const int row = j == KT ? K : j - (KT - K);
    if (row < 0) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) part[threadIdx.y][threadIdx.x][v] = j == KT ? db[v] : dw[j < KT ? j : 0][v];
    __syncthreads();
    for (int k = threadIdx.y * 32 + threadIdx.x; k < 32 * V; k += 32 * kBwdY) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < kBwdY; ++r) s += part[r][k / V][k % V];
      const int col = d - (int)threadIdx.x * V + k;
      if (col < c.D) ws[(int64_t)row * c.D + col] = s;
    }
    __syncthreads();
  }
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

bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Whether every row of every tensor can be read V elements at a time.
bool vec_ok(const ConvSeqArgs& c, int V, int es) {
  const int bytes = V * es;
  for (int64_t s : {c.sx.b, c.sx.t, c.sy.b, c.sy.t, (int64_t)c.D})
    if (s % V != 0) return false;
  for (const void* p : {c.x, c.w, c.bias, (const void*)c.y, c.state_in, (const void*)c.state_out, c.dy, c.dstate_out,
                        (const void*)c.dx, (const void*)c.dstate_in})
    if (!aligned(p, bytes)) return false;
  return true;
}

template <typename T, int V, int KT, int kRows>
cudaError_t fwd_k(const ConvSeqArgs& c, const LaunchArgs& a, const DeviceInfo& dev) {
  // batches of kRows tokens a thread walks: one while that leaves the GPU short of threads
  const int dblocks = (c.D + 32 * V - 1) / (32 * V);
  const int64_t batches = (c.T + kRows - 1) / kRows;
  const int64_t warps = c.B * batches * dblocks;
  int64_t nb = 1;
  while (nb < 4 && warps / (2 * nb) >= (int64_t)dev.num_sms * 32) nb *= 2;
  const int64_t tiles = (batches + nb - 1) / nb;
  const int64_t grid = (c.B * tiles + kFwdY - 1) / kFwdY * dblocks;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_kernel(conv1d_fwd_kernel<T, V, KT, kRows>, dim3((unsigned)grid), dim3(32, kFwdY), 0, a, c, (int)nb, tiles,
                       dblocks);
}

// A single token is its own batch.
template <typename T, int V, int KT>
cudaError_t fwd_t(const ConvSeqArgs& c, const LaunchArgs& a, const DeviceInfo& dev) {
  return c.T == 1 ? fwd_k<T, V, KT, 1>(c, a, dev) : fwd_k<T, V, KT, 8>(c, a, dev);
}

template <typename T, int V>
cudaError_t fwd_v(const ConvSeqArgs& c, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (c.K) {
    case 1: return fwd_t<T, V, 1>(c, a, dev);
    case 2: return fwd_t<T, V, 2>(c, a, dev);
    case 3: return fwd_t<T, V, 3>(c, a, dev);
    case 4: return fwd_t<T, V, 4>(c, a, dev);
    default: return fwd_t<T, V, kMaxK>(c, a, dev);
  }
}

template <typename T>
cudaError_t fwd(const ConvSeqArgs& c, const LaunchArgs& a, const DeviceInfo& dev) {
  constexpr int V = 4;  // 8 channels of 16 bits leave too few warps: 53 us against 45 (2 x 16384 x 2048)
  if (vec_ok(c, V, sizeof(T))) return fwd_v<T, V>(c, a, dev);
  return fwd_v<T, 1>(c, a, dev);
}

int64_t bwd_tiles(int64_t T) { return (T + kBwdTile - 1) / kBwdTile; }

template <typename T, int V, int KT>
cudaError_t bwd_k(const ConvSeqArgs& c, const LaunchArgs& a) {
  const int dblocks = (c.D + 32 * V - 1) / (32 * V);
  const int64_t tiles = bwd_tiles(c.T), parts = c.B * tiles;
  if (parts * dblocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_kernel(conv1d_bwd_kernel<T, V, KT>, dim3((unsigned)(parts * dblocks)), dim3(32, kBwdY), 0, a,
                                c, tiles, dblocks);
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)(c.K + 1) * c.D;
  return launch_kernel(conv1d_dw_kernel<T>, dim3((unsigned)((n + 31) / 32)), dim3(32, kSumRows), 0, a, c, parts);
}

template <typename T, int V>
cudaError_t bwd_v(const ConvSeqArgs& c, const LaunchArgs& a) {
  switch (c.K) {
    case 1: return bwd_k<T, V, 1>(c, a);
    case 2: return bwd_k<T, V, 2>(c, a);
    case 3: return bwd_k<T, V, 3>(c, a);
    case 4: return bwd_k<T, V, 4>(c, a);
    default: return bwd_k<T, V, kMaxK>(c, a);
  }
}

template <typename T>
cudaError_t bwd(const ConvSeqArgs& c, const LaunchArgs& a) {
  constexpr int V = 4;  // 8 channels of 16 bits would need over 128 registers
  if (vec_ok(c, V, sizeof(T))) return bwd_v<T, V>(c, a);
  return bwd_v<T, 1>(c, a);
}

}  // namespace

int64_t conv1d_bwd_workspace_bytes(int64_t B, int64_t T, int D, int K) { return B * bwd_tiles(T) * (K + 1) * D * 4; }

cudaError_t conv1d_fwd_launch(const ConvSeqArgs& c, const LaunchArgs& a, const DeviceInfo& dev) {
  switch (a.dt) {
    case kF32: return fwd<float>(c, a, dev);
    case kF16: return fwd<__half>(c, a, dev);
    default: return fwd<__nv_bfloat16>(c, a, dev);
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
