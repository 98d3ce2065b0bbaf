// 8-bit matrix product with scales for each row of both sides (gconv_matmul_q8):
//   y[m, n] = sx[m] * sw[n] * sum_k xq[m, k] * wq[n, k] (+ bias[n])
//
// Three kernels: few rows (M <= 8) on the integer dot-product instruction, bound
// by the bytes of wq; more rows on the tensor cores, from tiles that TMA copies; and
// the same from plain loads, for rows that TMA cannot take.
#include <algorithm>

#include "plan_cache.h"
#include "seq.h"
#include "seq_vec.cuh"
#include "tc_ptx.cuh"

namespace gconv {
namespace {

// scales and bias in fp32, one rounding
template <typename T>
__device__ __forceinline__ float finish(float acc, float sx, float sw, float bias) {
  return fmaf(acc * sx, sw, bias);
}

// ---------------------------------------------------------------------------
// Few rows: every byte of wq is read once, by a warp that takes R of its rows
// and all M rows of xq (those come from the first-level cache), 16 bytes a lane
// and step, four steps' reads together; the lanes' integer sums are added at the
// end.  KS: warps that share the K of their rows, where wq has few.
// 4 x 8192 x 2048 in a graph: 3.4 us with the weights in the second-level cache, 5.3 from
// memory (the bytes alone are 2.5), 5 rows from memory 8.1; the tensor-core kernel takes
// 8.2 at 16.  1 x 4096 x 4096 from memory 4.8, 8 x 4096 x 4096 9.2.  Launched
// back to back, R and KS 4 and 1 / 2 and 4 / 1 and 1 / 1 and 4, us:
//   1 x 8192 x 2048  4.5 / 5.8 / 4.2 / 8.7     2 x 4096 x 4096  6.5 / 4.9 / 5.5 / 5.9
//   1 x 4096 x 4096  6.4 / 5.7 / 4.6 / 5.4     4 x 2048 x 2048  4.0 / 2.4 / 3.6 / 3.4
//   1 x 1024 x 4096  5.9 / 3.3 / 3.4 / 2.6     4 x 8192 x 2048  4.8 / 6.0 / 6.3 / 9.6
//   8 x 4096 x 4096 (R 2)  7.1 / 8.8           8 x 1024 x 4096 (R 2)  7.0 / 3.1
// ---------------------------------------------------------------------------
constexpr int kFewRows = 8;
constexpr int kFewWarps = 4;

template <typename T, int MM, int R, int KS>
__global__ void __launch_bounds__(32 * kFewWarps) mmq_few_kernel(MatmulQ8Args a) {
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % KS;
  const int n0 = (blockIdx.x * (kFewWarps / KS) + warp / KS) * R, skip = (part * 32 + lane) * 16;
  const int8_t* w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = a.wq + (int64_t)(n0 + r < a.N ? n0 + r : a.N - 1) * a.K + skip;
  const int8_t* x = a.xq + skip;
  const int m_count = (int)a.M;
  int acc[R][MM];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MM; ++m) acc[r][m] = 0;
  grid_dependency_wait();
#pragma unroll 4
  for (int k = skip; k < a.K; k += 512 * KS) {
    int4 wv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      wv[r] = *reinterpret_cast<const int4*>(w[r]);
      w[r] += 512 * KS;
    }
#pragma unroll
    for (int m = 0; m < MM; ++m) {
      const int4 xv = *reinterpret_cast<const int4*>(x + (int64_t)(m < m_count ? m : 0) * a.K);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        acc[r][m] = __dp4a(wv[r].x, xv.x, acc[r][m]);
        acc[r][m] = __dp4a(wv[r].y, xv.y, acc[r][m]);
        acc[r][m] = __dp4a(wv[r].z, xv.z, acc[r][m]);
        acc[r][m] = __dp4a(wv[r].w, xv.w, acc[r][m]);
      }
    }
    x += 512 * KS;
  }
  // lane m * R + r keeps the sum of (r, m)
  int mine = 0;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MM; ++m) {
      const int sum = __reduce_add_sync(0xffffffffu, acc[r][m]);
      if (lane == m * R + r) mine = sum;
    }
  if constexpr (KS > 1) {
    __shared__ int sums[kFewWarps][32];
    sums[warp][lane] = mine;
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int k = 1; k < KS; ++k) mine += sums[warp + k][lane];
  }
  const int m = lane / R, n = n0 + lane % R;
  if (lane < MM * R && m < m_count && n < a.N) {
    const float b = a.bias ? Elem<T>::to_f32(static_cast<const T*>(a.bias)[n]) : 0.f;
    static_cast<T*>(a.y)[m * a.ys + n] = Elem<T>::from_f32(finish<T>((float)mine, a.sx[m], a.sw[n], b));
  }
}

// ---------------------------------------------------------------------------
// Tensor cores.  The 8-bit integer instruction is many times slower than the
// 16-bit one on this chip, and every 8-bit integer is exact in binary16, so the
// operands are widened on chip and multiplied as binary16 with fp32 sums: the
// bytes in memory stay 8-bit, the products exact.
//
// An output tile is 128 rows of wq (the instruction's M) x BX rows of xq (its
// N).  One persistent block an SM, its warps specialised:
//   warp 0        TMA copies of 128-byte pieces (K = 128) of the tile's rows
//   warps 6 ...   teams of six, each with every kTeams-th step of K = 64: four warps
//                 widen the rows of wq into tensor memory (a lane is a row), and
//                 all six, evenly loaded, those of xq into a second ring, in the
//                 128-byte-swizzled layout
//   warp 1        issues the instructions (four of K = 16 a step), their first
//                 operand in tensor memory
//   warps 2 ... 5  read the accumulators (one of two) from tensor memory, scale,
//                 add the bias, round and store; a lane is a row of wq, so a
//                 warp stores 32 neighbouring columns of a row of y.
// What bounds a large product is the bytes through shared memory: a step of K = 64
// copies in and reads 64 (128 + BX) bytes and writes and multiplies 128 BX, 608
// cycles at 128 bytes a cycle for BX = 160, and takes 296 ns = 607 cycles: 8192 x
// 8192 x 2048 in 212 us, 1297 TFLOP/s, 68% of the measured binary16 rate.  With
// both widened operands in shared memory it took 314 us.
// A step's way through a warp (wait, read, widen, write, fence, signal) is long
// next to its work; kTeams steps are on theirs together.  A team owns its stage
// of the second ring and of tensor memory, and the first ring holds a multiple of
// kTeams / 2 stages (a stage is two steps), so that a stage is always the same
// two teams': a team sees every phase of every barrier it waits on.  (A waiter
// that skipped one could take an older phase for its own.)
// SPLIT: where there are fewer tiles than SMs, a cluster of p.split blocks shares
// one, each with a part of K.  Each leaves its sums in its own shared memory, in the
// first ring's place, and adds its share of the rows over all blocks, in their order.
// ANY: rows that TMA cannot take (K or an address off 16 bytes).  The teams read them
// from memory, aligned words joined by shifts; rows of xq go straight into the second
// ring, rows of wq through a place of their warp's.  In a graph, us, against 64 x 64
// tiles of integer dot products: 1 x 2048 x 2047 8.1 / 108, 512 x 2001 x 2003 27 / 147,
// 2048 x 4001 x 2005 107 / 438, 8192 x 8192 x 2049 794 / 3283; bound by the
// instructions that fetch and join words.
// Tensor memory is taken before the wait for the kernel before.  That cannot keep it
// from a block that the wait is for: a block here has 960 threads of at least 61 registers, all
// but 4,096 of an SM's, and every other kernel that takes tensor memory needs more.
// ---------------------------------------------------------------------------
constexpr int kTeams = 4, kWideW = 4, kWideX = 2, kTeamWarps = kWideW + kWideX, kConvWarp0 = 6;
constexpr int kTcThreads = 32 * (kConvWarp0 + kTeams * kTeamWarps);
constexpr int kBatch = 4;  // 8-row groups whose reads a warp has in flight
constexpr int kMaxRing = 12;
constexpr int kStageBytes = 32 * 64;  // a warp's place for its rows of wq, where TMA cannot bring them
constexpr int kMaxShare = 8;               // blocks that share a tile: a portable cluster
constexpr int kRowsW = 128;
constexpr int kMaxBX = 160;                // more leaves the first ring two stages: 430 ns a step instead of 296
constexpr int kWideCol = 512 - 32 * kTeams;  // where the teams' stages begin: 32 columns of two binary16 values each

struct TcPlan {
  int BX, tiles_n, tiles_m, tiles, ksteps;
  int split, per;  // blocks that share a tile, and the copied stages (K = 128) of each
  int raw_stages;
  uint32_t raw_bytes, wide_bytes;  // of a stage
  uint32_t idesc;
  int* status;
  uint64_t limit;
};

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// An MMA (first operand in tensor memory) and a commit by one lane of the
// converged issuing warp, every lane of which executes them with the same operands.  (Issued under `if (lane == 0)`
// instead, a step of four took 600 cycles.)
__device__ __forceinline__ void mma_elect(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// Registers -> tensor memory: 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four signed bytes as binary16: with its sign bit flipped a byte is v + 128,
// which in the low bits of 1024 (0x6400) makes 1152 + v, exactly.
__device__ __forceinline__ void widen4(uint32_t b, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = b ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 rl = __hsub2(*reinterpret_cast<const __half2*>(&l), off);
  const __half2 rh = __hsub2(*reinterpret_cast<const __half2*>(&h), off);
  lo = *reinterpret_cast<const uint32_t*>(&rl);
  hi = *reinterpret_cast<const uint32_t*>(&rh);
}

// The four bytes at byte `at` of a buffer of `size` bytes, buf + at a multiple of 4; 0 outside it.
__device__ __forceinline__ uint32_t ld_word(const int8_t* buf, int64_t size, int64_t at) {
  if (at >= 0 && at + 4 <= size) return *reinterpret_cast<const uint32_t*>(buf + at);
  uint32_t v = 0;
  for (int j = 0; j < 4; ++j)
    if (at + j >= 0 && at + j < size) v |= (uint32_t)(uint8_t)buf[at + j] << (8 * j);
  return v;
}
// 64 bytes, from byte k, of 2 NI rows of K bytes at any address, as words: lane l has
// word l % 16 of the rows 2 i + l / 16.  `load` asks for the two aligned words around
// each (the second one is the next lane's; of the last lanes, the 17th of a row),
// `word` joins them; bytes past K and rows from `rows` on are 0.
template <int NI>
struct RowWords {
  uint32_t lo[NI], more;  // more: of row `lane`
  int by[2];  // bits to shift by, i even and odd: two rows further on is 2 K bytes
  int left;   // bytes of a row from this lane's word on
  bool whole;
  __device__ __forceinline__ void load(const int8_t* buf, int64_t rows, int64_t row0, int K, int k, int lane) {
    const int64_t size = rows * K, row = row0 + (lane >> 4);
    const int8_t* q = buf + row * K + k + 4 * (lane & 15);
    by[0] = (int)(reinterpret_cast<uintptr_t>(q) & 3) * 8;
    by[1] = (int)(reinterpret_cast<uintptr_t>(q + 2 * K) & 3) * 8;
    left = K - k - 4 * (lane & 15);
    // every row lives, has 64 bytes, and neither it nor its neighbouring words begin or end the buffer
    whole = row0 + 2 * NI <= rows && k + 64 <= K && row0 * K + k >= 4 && (row0 + 2 * NI - 1) * K + k + 68 <= size;
    if (whole) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t* at = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(q + (int64_t)(2 * i) * K) & ~(uintptr_t)3);
        lo[i] = *at;
      }
      const uintptr_t last = reinterpret_cast<uintptr_t>(buf + (row0 + (lane & (2 * NI - 1))) * K + k + 64);
      more = *reinterpret_cast<const uint32_t*>(last & ~(uintptr_t)3);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int64_t at = q - buf + (int64_t)(2 * i) * K - by[i & 1] / 8;
        const bool in = row + 2 * i < rows && left > -4;  // the lane before may need it for its last bytes
        lo[i] = in ? ld_word(buf, size, at) : 0u;
      }
      const int64_t end = (row0 + (lane & (2 * NI - 1))) * K + k + 64;
      more = row0 + (lane & (2 * NI - 1)) < rows && k + 60 < K
                 ? ld_word(buf, size, end - (int64_t)(reinterpret_cast<uintptr_t>(buf + end) & 3)) : 0u;
    }
  }
  __device__ __forceinline__ uint32_t word(int i, int lane) const {
    const uint32_t down = __shfl_down_sync(0xffffffffu, lo[i], 1), last = __shfl_sync(0xffffffffu, more, 2 * i + (lane >> 4));
    const uint32_t v = __funnelshift_r(lo[i], (lane & 15) == 15 ? last : down, by[i & 1]);
    return whole || left >= 4 ? v : left <= 0 ? 0u : v & ((1u << (8 * left)) - 1u);
  }
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The four values at `at` (an address in this block's shared memory) of block `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster(uint32_t at, int rank) {
  uint32_t from;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(from) : "memory");
  return v;
}

template <typename T, bool SPLIT, bool ANY>
__global__ void __launch_bounds__(kTcThreads, 1)
mmq_tc_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, MatmulQ8Args a,
              TcPlan p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t raw_full[kMaxRing], raw_empty[kMaxRing], wide_full[kTeams], wide_empty[kTeams], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int failed;
  unsigned char* raw = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* wide = raw + p.raw_stages * p.raw_bytes;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int k = 0; k < p.raw_stages; ++k) {
      mbar_init(&raw_full[k], 1);
      mbar_init(&raw_empty[k], 2 * kTeamWarps);  // a stage is two steps
    }
    for (int k = 0; k < kTeams; ++k) {
      mbar_init(&wide_full[k], kTeamWarps);
      mbar_init(&wide_empty[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&acc_full[k], 1);
      mbar_init(&acc_empty[k], 4);
    }
    mbar_init(&drain, 1);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(&tmem_slot, 512);
  allow_dependent_launch();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  // After a wait that ran out nothing waits or works any more; the block reaches its end.
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) {  // one thread
    if (mbar_try_wait(bar, parity)) return true;
    if (failed) return false;
    if (mbar_wait(bar, parity, p.limit)) return true;
    report(p.status, kDevTimeout, site);
    failed = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity, int site) {  // a converged warp, with one answer
    return __all_sync(0xffffffffu, wait(bar, parity, site));
  };
  const int first = SPLIT ? (int)blockIdx.x / p.split : (int)blockIdx.x, rank = SPLIT ? (int)blockIdx.x - first * p.split : 0;
  const int my_tiles = SPLIT ? 1 : first < p.tiles ? (p.tiles - 1 - first) / (int)gridDim.x + 1 : 0;
  const int kfirst = SPLIT ? rank * p.per : 0;  // in copied stages
  const int ksteps = SPLIT ? min(2 * p.per, p.ksteps - 2 * kfirst) : p.ksteps;
  const int steps = my_tiles * ksteps;
  const uint32_t raw_w = kRowsW * 128u;  // where xq's part of a copied stage begins
  if (warp == 0) {
    if (!ANY && lane == 0) {
      grid_dependency_wait();
      int step = 0;
      for (int i = 0; i < my_tiles && !failed; ++i) {
        const int tile = first + i * (int)gridDim.x;
        const int tm = tile / p.tiles_n, tn = tile - tm * p.tiles_n;
        for (int k = 0; k < ksteps / 2; ++k, ++step) {
          const int st = step % p.raw_stages, use = step / p.raw_stages;
          if (use > 0 && !wait(&raw_empty[st], (uint32_t)(use - 1) & 1u, 80)) break;
          unsigned char* to = raw + st * p.raw_bytes;
          mbar_arrive_expect_tx(&raw_full[st], p.raw_bytes);
          tma_load_2d(to, &wmap, &raw_full[st], (kfirst + k) * 128, tn * kRowsW);
          tma_load_2d(to + raw_w, &xmap, &raw_full[st], (kfirst + k) * 128, tm * p.BX);
        }
      }
      // no copy is in flight when the block ends, also after a wait that ran out
      for (int back = step < p.raw_stages ? 0 : step - p.raw_stages; back < step; ++back)
        mbar_wait(&raw_full[back % p.raw_stages], (uint32_t)(back / p.raw_stages) & 1u, p.limit);
    }
  } else if (warp == 1) {
    const uint32_t wide_at = smem_u32(wide);
    int st = 0;
    uint32_t parity = 0;
    for (int i = 0; i < my_tiles; ++i) {
      const int acc = i & 1;
      if (i >= 2 && !wait_warp(&acc_empty[acc], (uint32_t)((i >> 1) - 1) & 1u, 81)) break;
      tc::fence_after_sync();
      bool ok = true;
      for (int k = 0; k < ksteps; ++k) {
        ok = wait_warp(&wide_full[st], parity, 82);
        if (!ok) break;
        tc::fence_after_sync();
        const uint64_t xd = tc::smem_desc_sw128(wide_at + st * p.wide_bytes);
#pragma unroll
        for (int q = 0; q < 4; ++q)  // K = 16 is 8 columns, and 32 bytes: 2 in the descriptor's address units
          mma_elect(tmem + acc * kMaxBX, tmem + kWideCol + st * 32 + 8 * q, xd + 2 * q, p.idesc, k > 0 || q > 0);
        commit_elect(&wide_empty[st]);
        if (++st == kTeams) st = 0, parity ^= 1u;
      }
      if (!ok) break;
      commit_elect(&acc_full[acc]);
    }
    // every instruction has finished before the block gives its tensor memory back
    commit_elect(&drain);
    if (!mbar_wait(&drain, 0, p.limit)) report(p.status, kDevTimeout, 83);
  } else if (SPLIT && warp < kConvWarp0) {
    // this block's sums, [row of xq][row of wq]; the first ring's copies have all been read
    const int quarter = warp & 3, tm = first / p.tiles_n;
    const int64_t m0 = (int64_t)tm * p.BX;
    const int rows = a.M - m0 < p.BX ? (int)(a.M - m0) : p.BX;
    if (wait_warp(&acc_full[0], 0, 84)) {
      tc::fence_after_sync();
      float* part = reinterpret_cast<float*>(raw) + quarter * 32 + lane;
      for (int c = 0; c < rows; c += 16) {
        uint32_t v[16];
        tc::tmem_ld16(tmem + c + ((uint32_t)quarter << 21), v);
        tc::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * kRowsW] = __uint_as_float(v[j]);
      }
    }
  } else if (warp < kConvWarp0) {
    grid_dependency_wait();
    const int quarter = warp & 3;  // the tensor-memory lanes a warp may read
    for (int i = 0; i < my_tiles; ++i) {
      const int tile = first + i * (int)gridDim.x;
      const int tm = tile / p.tiles_n, tn = tile - tm * p.tiles_n, acc = i & 1;
      const int n = tn * kRowsW + quarter * 32 + lane;
      const bool live = n < a.N;
      const float sw = live ? a.sw[n] : 0.f;
      const float bias = live && a.bias ? Elem<T>::to_f32(static_cast<const T*>(a.bias)[n]) : 0.f;
      if (!wait_warp(&acc_full[acc], (uint32_t)(i >> 1) & 1u, 84)) break;
      tc::fence_after_sync();
      const int64_t m0 = (int64_t)tm * p.BX;
      const int rows = a.M - m0 < p.BX ? (int)(a.M - m0) : p.BX;
      T* y = static_cast<T*>(a.y) + m0 * a.ys + n;
      for (int c = 0; c < rows; c += 32) {
        // lane j holds the scale of row c + j
        const float scales = c + lane < rows ? a.sx[m0 + c + lane] : 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (c + 16 * h >= rows) break;
          uint32_t v[16];
          tc::tmem_ld16(tmem + acc * kMaxBX + c + 16 * h + ((uint32_t)quarter << 21), v);
          tc::tmem_ld_wait();
          const bool whole = c + 16 * h + 16 <= rows;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float sx = __shfl_sync(0xffffffffu, scales, 16 * h + j);
            if (live && (whole || c + 16 * h + j < rows)) *y = Elem<T>::from_f32(finish<T>(__uint_as_float(v[j]), sx, sw, bias));
            y += a.ys;
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
    }
  } else {
    // Rows of 128 bytes, piece c of row r at c ^ (r % 8), in both rings: eight rows'
    // pieces of a quarter warp lie in different banks.
    const int team = (warp - kConvWarp0) / kTeamWarps, role = (warp - kConvWarp0) % kTeamWarps;
    const int half = team & 1;  // kTeams is even: the half of a copied stage is the team's
    const int quarter = warp & 3, row = quarter * 32 + lane;  // wq: four consecutive warps have all four quarters
    const int r8 = lane & 7, c = lane >> 3, groups = p.BX / 8;
    const uint32_t from = r8 * 128 + (((4 * half + c) ^ r8) << 4);
    const uint32_t to0 = r8 * 128 + (((2 * c) ^ r8) << 4), to1 = r8 * 128 + (((2 * c + 1) ^ r8) << 4);
    unsigned char* dst = wide + team * p.wide_bytes;
    const uint32_t tdst = tmem + kWideCol + team * 32 + ((uint32_t)quarter << 21);
    // 8-row groups of xq: the warps with rows of wq (four groups' worth of work
    // each) take `extra`, the other two share the rest
    const int even = (kRowsW / 8 + groups + kTeamWarps / 2) / kTeamWarps - 4, extra = even > 0 ? even : 0;
    const int rest = groups - kWideW * extra, first_half = (rest + 1) / 2;
    const int my_first = role < kWideW ? role * extra : kWideW * extra + (role - kWideW) * first_half;
    const int my_end = role < kWideW ? my_first + extra : role == kWideW ? my_first + first_half : groups;
    int rs = team / 2;
    uint32_t raw_parity = 0, wide_parity = 1;
    unsigned char* const mine = raw + (team * kWideW + role) * kStageBytes;  // of a warp with rows of wq, where ANY
    if (ANY) grid_dependency_wait();
    for (int step = team; step < steps; step += kTeams) {
      if (!ANY && !wait_warp(&raw_full[rs], raw_parity, 85)) break;
      int64_t any_m = 0;  // where ANY: the tile's first row of xq and of wq, and the step's first byte of a row
      int any_n = 0, any_k = 0;
      RowWords<16> any_w;
      if constexpr (ANY) {
        const int i = step / ksteps, tile = first + i * (int)gridDim.x, tm = tile / p.tiles_n;
        any_m = (int64_t)tm * p.BX, any_n = (tile - tm * p.tiles_n) * kRowsW, any_k = 128 * kfirst + 64 * (step - i * ksteps);
        if (role < kWideW) any_w.load(a.wq, a.N, any_n + quarter * 32, a.K, any_k, lane);
      }
      if (step >= kTeams && !wait_warp(&wide_empty[team], wide_parity, 86)) break;
      const unsigned char* src = raw + rs * p.raw_bytes;
      if (role < kWideW) {
        uint4 in[4];
        if constexpr (ANY) {
          // 32 rows of 64 bytes through the warp's own place, piece c of row r at c ^ (r / 2 % 4)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = 2 * i + (lane >> 4), w = lane & 15;
            *reinterpret_cast<uint32_t*>(mine + r * 64 + (((w >> 2) ^ (i & 3)) << 4) + (w & 3) * 4) =
                any_w.word(i, lane);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) in[k] = *reinterpret_cast<const uint4*>(mine + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4));
        } else {
          const unsigned char* at = src + row * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) in[k] = *reinterpret_cast<const uint4*>(at + (((4 * half + k) ^ (row & 7)) << 4));
        }
        tc::fence_after_sync();  // the instructions that read the stage before
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[16];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            widen4(in[2 * h + k].x, o[8 * k], o[8 * k + 1]);
            widen4(in[2 * h + k].y, o[8 * k + 2], o[8 * k + 3]);
            widen4(in[2 * h + k].z, o[8 * k + 4], o[8 * k + 5]);
            widen4(in[2 * h + k].w, o[8 * k + 6], o[8 * k + 7]);
          }
          tmem_st16(tdst + 16 * h, o);
        }
      }
      if constexpr (ANY) {
        for (int g0 = my_first; g0 < my_end; g0 += 2) {  // sixteen rows at a time
          RowWords<8> x;
          x.load(a.xq, a.M, any_m + g0 * 8, a.K, any_k, lane);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = (2 * i + (lane >> 4)) & 7, w = lane & 15;
            uint2 o;
            widen4(x.word(i, lane), o.x, o.y);
            if (g0 + i / 4 < my_end)
              *reinterpret_cast<uint2*>(dst + (g0 + i / 4) * 1024 + r * 128 + (((w >> 1) ^ r) << 4) + (w & 1) * 8) = o;
          }
        }
      }
      src += raw_w + from;
      for (int g0 = ANY ? my_end : my_first; g0 < my_end; g0 += kBatch) {
        uint4 in[kBatch];
#pragma unroll
        for (int g = 0; g < kBatch; ++g)
          if (g0 + g < my_end) in[g] = *reinterpret_cast<const uint4*>(src + (g0 + g) * 1024);
#pragma unroll
        for (int g = 0; g < kBatch; ++g)
          if (g0 + g < my_end) {
            uint4 o0, o1;
            widen4(in[g].x, o0.x, o0.y);
            widen4(in[g].y, o0.z, o0.w);
            widen4(in[g].z, o1.x, o1.y);
            widen4(in[g].w, o1.z, o1.w);
            *reinterpret_cast<uint4*>(dst + (g0 + g) * 1024 + to0) = o0;
            *reinterpret_cast<uint4*>(dst + (g0 + g) * 1024 + to1) = o1;
          }
      }
      fence_proxy_async_smem();
      if (role < kWideW) {
        tmem_st_wait();
        tc::fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) {
        if (!ANY) mbar_arrive(&raw_empty[rs]);
        mbar_arrive(&wide_full[team]);
      }
      wide_parity ^= 1u;
      rs += kTeams / 2;
      if (rs >= p.raw_stages) rs -= p.raw_stages, raw_parity ^= 1u;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_relinquish();
    tc::tmem_dealloc(tmem, 512);
  }
  if constexpr (SPLIT) {
    grid_dependency_wait();
    const int tm = first / p.tiles_n, tn = first - tm * p.tiles_n;
    const int64_t m0 = (int64_t)tm * p.BX;
    const int rows = a.M - m0 < p.BX ? (int)(a.M - m0) : p.BX;
    const int n = tn * kRowsW + 4 * lane;  // a warp takes whole rows, a lane four columns
    const bool whole = n + 4 <= a.N && a.ys % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & (4 * sizeof(T) - 1)) == 0;
    float sw[4], bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sw[e] = n + e < a.N ? a.sw[n + e] : 0.f;
      bias[e] = n + e < a.N && a.bias ? Elem<T>::to_f32(static_cast<const T*>(a.bias)[n + e]) : 0.f;
    }
    T* y = static_cast<T*>(a.y) + m0 * a.ys + n;
    const uint32_t part = smem_u32(raw) + (uint32_t)lane * 16u;
    cluster_sync();  // every block's sums are there
    for (int c = rank + warp * p.split; c < rows; c += kTcThreads / 32 * p.split) {
      const float sx = a.sx[m0 + c];
      float4 v[kMaxShare];
#pragma unroll
      for (int k = 0; k < kMaxShare; ++k)
        if (k < p.split) v[k] = ld_cluster(part + (uint32_t)c * (kRowsW * 4), k);
      float o[4] = {};
#pragma unroll
      for (int k = 0; k < kMaxShare; ++k)
        if (k < p.split) o[0] += v[k].x, o[1] += v[k].y, o[2] += v[k].z, o[3] += v[k].w;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = finish<T>(o[e], sx, sw[e], bias[e]);
      if (whole) {
        st_raw<T, 4>(y + c * a.ys, narrow<T, 4>(o));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.N) y[c * a.ys + e] = Elem<T>::from_f32(o[e]);
      }
    }
    cluster_sync();  // no block leaves while another reads its sums
  }
}

// Blocks of clusters of `split` that run at once, one an SM: with 152 SMs the device
// reports 152 of 2, 138 of 3, 144 of 4, 140 of 5, 138 of 6, 105 of 7 and 120 of 8.
int share_sms(int split, int sms) { return split <= 2 ? sms : split <= 6 ? sms * 9 / 10 : sms * 3 / 4; }

// Plan: BX, the rows of xq in a tile.  A step of a tile took, in ns: 16 ... 64 rows
// 200-230 (a team's way through a step), 80: 230, 96: 245, 112: 257, 128: 267,
// 144: 281, 160: 296 (the bytes through shared memory) over products of 64 x 8192
// x 2048 to 8192 x 8192 x 2048; 157 + BX follows that from 64 on.  The grid takes
// ceil(tiles / SMs) rounds of tiles.
// Sharing a tile costs 1.5 us and 22 ns a row more than its steps (longer rows to
// begin with, and the sums' way through the other blocks' shared memory).  In a graph,
// us, one block a tile / shared: 16 x 2048 x 2048 9.4 / 6.1 (six blocks), 16 x 1024 x
// 4096 15.6 / 6.3 (eight), 64 x 4096 x 4096 16.3 / 9.4 (four), 128 x 2048 x 2048 10.0 /
// 7.5, 16 x 8192 x 2048 9.5 / 8.2 (two); not taken, 128 x 4096 x 1024 6.4 / 8.6 and 512
// x 2048 x 2048 10.0 / 11.2.
// any: for the kernel that does without TMA, whose sizes and alignment are free.
bool tc_plan(const MatmulQ8Args& m, const DeviceInfo& dev, TcPlan* p, bool any = false) {
  if (!any && (m.K % 16 != 0 || (reinterpret_cast<uintptr_t>(m.xq) & 15) || (reinterpret_cast<uintptr_t>(m.wq) & 15)))
    return false;
  const int64_t tiles_n = (m.N + kRowsW - 1) / kRowsW;
  const int stages = (m.K + 127) / 128;
  int64_t best = -1;
  for (int bx = 16; bx <= kMaxBX; bx += 16) {
    const int64_t tiles_m = (m.M + bx - 1) / bx;
    if (bx > 16 && m.M <= bx - 16) break;
    const int64_t tiles = tiles_m * tiles_n, rounds = (tiles + dev.num_sms - 1) / dev.num_sms;
    if (tiles > 0x7fffffff) continue;
    for (int split = 1; split <= std::min(kMaxShare, stages); ++split) {
      if (split > 1 && (split == 7 || tiles * split > share_sms(split, dev.num_sms))) continue;
      const int per = (stages + split - 1) / split;
      if (split > 1 && (per * (split - 1) >= stages || bx * 512 > 2 * (kRowsW + bx) * 128)) continue;
      const int64_t cost = rounds * (2 * per) * std::max(218, 157 + bx) + (split > 1 ? 1500 + 22 * bx : 0);
      if (best < 0 || cost < best) {
        best = cost;
        p->BX = bx, p->tiles_m = (int)tiles_m, p->tiles_n = (int)tiles_n, p->tiles = (int)tiles;
        p->split = split, p->per = per;
      }
    }
  }
  if (best < 0) return false;
  p->ksteps = 2 * stages;
  if ((int64_t)(p->tiles / dev.num_sms + 1) * p->ksteps > 0x7fffffff) return false;
  p->raw_bytes = (uint32_t)(kRowsW + p->BX) * 128;
  p->wide_bytes = (uint32_t)p->BX * 128;
  p->idesc = tc::idesc_f16(false, kRowsW, p->BX);
  if (any) {  // no ring: the warps' places, and later a shared tile's sums
    p->raw_stages = 1, p->raw_bytes = (uint32_t)std::max(kTeams * kWideW * kStageBytes, p->BX * 512);
    return true;
  }
  const int room = dev.max_smem_optin - 1024 - 1024;  // alignment, barriers
  p->raw_stages = std::min(kMaxRing, (room - kTeams * (int)p->wide_bytes) / (int)p->raw_bytes) / (kTeams / 2) * (kTeams / 2);
  return p->raw_stages >= kTeams / 2;
}

bool byte_map(CUtensorMap* map, const int8_t* p, int64_t rows, int K, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)K, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)K};
  const uint32_t box[2] = {128, (uint32_t)box_rows}, ones[2] = {1, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, dims, strides, box, ones, CU_TENSOR_MAP_SWIZZLE_128B) ==
         CUDA_SUCCESS;
}

template <auto kernel, typename... Args>
cudaError_t launch_tc(int blocks, size_t smem, int cluster, const LaunchArgs& a, const DeviceInfo& dev, Args&&... args) {
  static SmemAttr most;
  const cudaError_t e = most.ensure(kernel, dev.device, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename T, int MM, int R, int KS>
cudaError_t launch_few(const MatmulQ8Args& m, const LaunchArgs& a) {
  const int per = kFewWarps / KS * R;
  return launch_kernel(mmq_few_kernel<T, MM, R, KS>, dim3((unsigned)((m.N + per - 1) / per)), dim3(32 * kFewWarps), 0, a, m);
}

template <typename T>
cudaError_t launch(const MatmulQ8Args& m, const LaunchArgs& a, const DeviceInfo& dev) {
  const bool vec = m.K % 16 == 0 && !(reinterpret_cast<uintptr_t>(m.xq) & 15) && !(reinterpret_cast<uintptr_t>(m.wq) & 15);
  if (m.M <= kFewRows && vec) {
    // rows of wq enough to fill the GPU with whole ones, or warps that share a row's K
    const bool share = m.K >= 2048 && m.N <= (m.M == 1 ? 8 : m.M <= 4 ? 28 : 16) * dev.num_sms;
    if (m.M == 1) return share ? launch_few<T, 1, 1, 4>(m, a) : launch_few<T, 1, 1, 1>(m, a);
    if (m.M == 2) return share ? launch_few<T, 2, 2, 4>(m, a) : launch_few<T, 2, 4, 1>(m, a);
    if (m.M <= 4) return share ? launch_few<T, 4, 2, 4>(m, a) : launch_few<T, 4, 4, 1>(m, a);
    return share ? launch_few<T, 8, 2, 4>(m, a) : launch_few<T, 8, 2, 1>(m, a);
  }
  TcPlan p = {};
  CUtensorMap wmap = {}, xmap = {};
  const bool tma = vec && tc_plan(m, dev, &p) && byte_map(&wmap, m.wq, m.N, m.K, kRowsW) && byte_map(&xmap, m.xq, m.M, m.K, p.BX);
  if (!tma && !tc_plan(m, dev, &p, true)) return cudaErrorInvalidConfiguration;  // more tiles than 31 bits count
  p.status = a.status;
  p.limit = a.wait_limit_ns;
  const size_t smem = 1024 + (size_t)p.raw_stages * p.raw_bytes + (size_t)kTeams * p.wide_bytes;
  const int blocks = p.split > 1 ? p.tiles * p.split : std::min(p.tiles, dev.num_sms);
  if (tma)
    return p.split > 1 ? launch_tc<mmq_tc_kernel<T, true, false>>(blocks, smem, p.split, a, dev, wmap, xmap, m, p)
                       : launch_tc<mmq_tc_kernel<T, false, false>>(blocks, smem, p.split, a, dev, wmap, xmap, m, p);
  return p.split > 1 ? launch_tc<mmq_tc_kernel<T, true, true>>(blocks, smem, p.split, a, dev, wmap, xmap, m, p)
                     : launch_tc<mmq_tc_kernel<T, false, true>>(blocks, smem, p.split, a, dev, wmap, xmap, m, p);
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
