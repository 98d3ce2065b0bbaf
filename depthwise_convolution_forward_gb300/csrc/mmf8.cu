// Product of 8-bit floating-point matrices with block scales (gconv_matmul_f8):
//   y[m, n] = sum_kb sx[kb, m] sw[kb, n / w_rows] sum_{k in kb} xq[m, k] wq[n, k] (+ bias[n])
//
// The tensor cores take the bytes as they lie (kind::f8f6f4), one block of K = 128 at a time: a
// tile's sums over one block go to tensor memory, one of two buffers, and two warpgroups take them from
// there, times the block's scales, into fp32 sums in registers while the next block is multiplied.
#include <algorithm>

#include "plan_cache.h"
#include "seq_vec.cuh"
#include "ssm.h"
#include "tc_ptx.cuh"

namespace gconv {
namespace {

// ---------------------------------------------------------------------------
// An output tile is rows of the instruction's first operand (tensor-memory lanes) x BN rows of its second
// (columns).  Two forms:
//   pair   a cluster of two blocks on a tile of 256 rows of xq x 256 of wq, multiplied by one
//          instruction for both SMs (cta_group::2): each copies its 128 rows of xq and half of those of wq, so
//          that 32 KB a step come to an SM instead of 48 (which 64 bytes a cycle, an SM's way in, take 770 cycles
//          for, and the instructions 512).  A lane is a row of y; tiles go out through shared memory by TMA.
//   SWAP   first operand 128 rows of wq, second BN = 16 ... 128 of xq, for fewer rows: a lane is a column of
//          y, and a warp stores 32 neighbouring ones.  Where there are fewer tiles than SMs a
//          cluster of p.split blocks shares one, each with a part of K; they leave their sums in
//          shared memory and add them over the blocks in order.
// COLS: the second operand has a scale for each row (a column here); else one for all 128 columns of a
// warpgroup.
//
// Warps 0 ... 7 are the two warpgroups (columns are halved between them), warp 8 copies (TMA, 128-byte swizzle), warp 9
// issues the instructions, warp 10 copies the scales into a ring, without waiting for them (read by the lanes that use
// them they took a step 700 cycles).  In the pair form a lane holds 128 sums: its warpgroups take registers from the
// third one (kSumRegs and kRestRegs together are the block's registers at launch, 168 a thread).
//
// Measured, us: pairs 8192 x 8192 x 2048 bf16 128 (2155 TFLOP/s; one block on 128 x 256 took 144 to 156, sums read 32
// columns a time and lane-read scales 208 to 249), 4096 x 4096 x 4096 69 (2002), with a scale for each row of wq 4096 x
// 2048 x 8192 fp32 102.  A step takes a pair 520 ns, in which the instructions are at work half of the time (47 to 53%
// of the tensor pipe) and 44% of the issue slots are taken, some 200 instructions a summing warp, where 64 packed fused
// products and additions and 4 loads are the work: neither is full, and what the rest is has not been measured.  A
// buffer of sums is given back whole, so that the next but one step's instructions wait for most of a step's reads.
// With a scale for each column a step takes 800 ns; every summing warp then reads 128 of them from shared memory, 32
// loads of 16 bytes that all lanes make alike, which has not been measured apart.  Few rows: 4 x 8192 x 2048 8.3, 64
// rows 9.9, by the latency of a step's way through copy, instruction and sums (300 ns; eight of sixteen steps a block,
// two blocks a tile), the sums' way between the blocks, and the launch.
// ---------------------------------------------------------------------------
constexpr int kRowsA = 128;
constexpr int kStep = GCONV_F8_BLOCK;  // K of a step, in bytes
constexpr int kMaxStages = 12;
constexpr int kScaleRing = 8;
constexpr int kFirstCopies = 2;  // steps asked for before the block is set up (a ring has at least as many stages)
constexpr int kMaxSplit = 8;
constexpr int kF8Threads = 384;
constexpr int kSumRegs = 224, kRestRegs = 56;
static_assert(2 * kSumRegs + kRestRegs == 3 * 168, "a warpgroup would wait for registers for ever");
constexpr int kOutBytes = 2 * 32 * 128;  // of a warp's rows of y on their way out: two pieces of 32 rows x 128 bytes

struct F8Plan {
  int BN, tiles_b, tiles, ksteps;
  int split, per;  // blocks that share a tile, steps of each
  int half;        // columns of the first warpgroup
  int stages;
  bool y_map;      // rows of y by TMA
  uint32_t stage_bytes, idesc;
  DType dt;
  int* status;
  uint64_t limit;
};

// Steps go through a ring's stages in turn, a barrier each.  After `steps` of them, the first one whose stage no later one
// has taken, so that nobody has waited for what it leaves behind; its stage and its barrier's phase.
struct OpenSteps {
  int from, stage;
  uint32_t phase;
};
__host__ __device__ constexpr OpenSteps open_steps(int steps, int stages) {
  const int from = steps > stages ? steps - stages : 0;
  return {from, from % stages, (uint32_t)(from / stages) & 1u};
}

// One side of the product.
struct Side {
  const float* scale;
  int64_t stride, rows;
  int group;  // rows with one scale
};

__device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// The same for a block of a pair: its bytes count for the barrier at `bar`, which may be the other block's.
__device__ __forceinline__ void load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
// An MMA and a commit by one lane of the converged issuing warp.  PAIR: for both blocks; the
// commit arrives in both.
template <bool PAIR>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
template <bool PAIR>
__device__ __forceinline__ void commit_one(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t.reg .b16 m;\n\t"
        "mov.b16 m, 3;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(smem_u32(bar))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void take_tmem(uint32_t* slot, uint32_t columns) {
  if constexpr (PAIR)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(columns) : "memory");
  else
    tc::tmem_alloc(slot, columns);
}
template <bool PAIR>
__device__ __forceinline__ void return_tmem(uint32_t at, uint32_t columns) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
  } else {
    tc::tmem_relinquish();
    tc::tmem_dealloc(at, columns);
  }
}
// A scale to shared memory, or 0.
__device__ __forceinline__ void copy_scale(float* to, const float* from, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 4 : 0) : "memory");
}
// The address of `bar` in block `rank` of the cluster, and an arrival there.  Relaxed: what it
// orders is reads of tensor memory, which tcgen05.wait and the fence before it have finished; with
// release.cluster it took 900 cycles.
__device__ __forceinline__ uint32_t peer_of(uint64_t* bar, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(bar)), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A number for another block of the cluster: to its shared memory at `to`, and an arrival at its barrier `bar`.
__device__ __forceinline__ void tell(int* to, uint64_t* bar, int value, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(to)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(value) : "memory");
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_of(bar, rank)) : "memory");
}
// Tensor memory -> registers: 32 lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t at, int rank) {
  uint32_t from;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(from) : "memory");
  return v;
}
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// y's element type is known at run time only: the sums' loop is by far the larger part.
__device__ __forceinline__ void store_one(void* y, int64_t at, float v, DType dt) {
  if (dt == kF32)
    static_cast<float*>(y)[at] = v;
  else if (dt == kF16)
    static_cast<__half*>(y)[at] = Elem<__half>::from_f32(v);
  else
    static_cast<__nv_bfloat16*>(y)[at] = Elem<__nv_bfloat16>::from_f32(v);
}
__device__ __forceinline__ float load_one(const void* p, int64_t at, DType dt) {
  return dt == kF32   ? static_cast<const float*>(p)[at]
         : dt == kF16 ? Elem<__half>::to_f32(static_cast<const __half*>(p)[at])
                      : Elem<__nv_bfloat16>::to_f32(static_cast<const __nv_bfloat16*>(p)[at]);
}

template <bool SWAP, bool COLS>
__global__ void __launch_bounds__(kF8Threads, 1)
mmf8_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
            const __grid_constant__ CUtensorMap ymap, Side sa, Side sb, void* y, const void* bias, int64_t ys, F8Plan p) {
  constexpr bool PAIR = !SWAP;
  constexpr int NC = SWAP ? 64 : 128;  // columns of a warpgroup at most
  constexpr int kAcc = 512 / (2 * NC);  // buffers of sums: all of tensor memory
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[kAcc], acc_empty[kAcc], sc_full[kScaleRing], sc_empty[kScaleRing], drain, told;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int failed;
  __shared__ int others;  // PAIR, first block: steps that the second one has copied
  unsigned char* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* const out = ring + p.stages * p.stage_bytes;              // PAIR: a warp's kOutBytes, on 1024 bytes
  unsigned char* const after = out + (PAIR ? 8 * kOutBytes : 0);
  constexpr int kScales = kRowsA + (COLS ? 2 * NC : 4);                    // of a step: the lanes', then the columns'
  float* const scales = reinterpret_cast<float*>(after);                   // [ring][kScales]
  float* const col_bias = scales + kScaleRing * kScales;                   // PAIR: [2 NC]
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int in_cluster = PAIR ? 2 : p.split;
  const int first = (int)blockIdx.x / in_cluster, rank = (int)blockIdx.x - first * in_cluster;
  const bool shared = SWAP && p.split > 1;
  const int stride = (int)gridDim.x / in_cluster;
  const int rows_a = PAIR ? 2 * kRowsA : kRowsA, rank_a = PAIR ? rank * kRowsA : 0;  // rows of a tile; this block's first
  const int my_tiles = first < p.tiles ? (p.tiles - 1 - first) / stride + 1 : 0;
  const int kfirst = PAIR ? 0 : rank * p.per, ksteps = min(p.per, p.ksteps - kfirst);
  const int total = my_tiles * ksteps;
  // The copying lane's place: the next step's stage, block of K and tile.
  int copied = 0, copy_st = 0, copy_k = 0, copy_a = first / p.tiles_b, copy_b = first - copy_a * p.tiles_b;
  auto copy = [&]() {  // the next step's
    unsigned char* to = ring + copy_st * p.stage_bytes;
    const int c = (kfirst + copy_k) * kStep;
    if constexpr (PAIR) {  // both blocks' bytes count in the first one, which multiplies
      if (rank == 0) mbar_arrive_expect_tx(&full[copy_st], 2 * p.stage_bytes);
      const uint32_t bar = peer_of(&full[copy_st], 0);
      load_2d_pair(to, &amap, bar, c, copy_a * rows_a + rank_a);
      load_2d_pair(to + kRowsA * kStep, &bmap, bar, c, copy_b * p.BN + rank * kRowsA);
    } else {
      mbar_arrive_expect_tx(&full[copy_st], p.stage_bytes);
      load_2d(to, &amap, &full[copy_st], c, copy_a * rows_a);
      load_2d(to + kRowsA * kStep, &bmap, &full[copy_st], c, copy_b * p.BN);
    }
    ++copied;
    if (++copy_st == p.stages) copy_st = 0;
    if (++copy_k == ksteps) {
      copy_k = 0;
      for (copy_b += stride; copy_b >= p.tiles_b; copy_b -= p.tiles_b) ++copy_a;
    }
  };
  if (threadIdx.x == 256) {
    for (int k = 0; k < p.stages; ++k) {
      mbar_init(&full[k], 1);
      mbar_init(&empty[k], 1);
    }
    for (int k = 0; k < kAcc; ++k) {
      mbar_init(&acc_full[k], 1);
      mbar_init(&acc_empty[k], PAIR ? 16 : 8);
    }
    for (int k = 0; k < kScaleRing; ++k) {
      mbar_init(&sc_full[k], 32);
      mbar_init(&sc_empty[k], 8);
    }
    mbar_init(&drain, 1);
    mbar_init(&told, 1);
    failed = 0;
    tma_prefetch_desc(&amap);
    tma_prefetch_desc(&bmap);
    fence_mbar_init();
    if constexpr (!PAIR) {  // the first copies need no other warp
      grid_dependency_wait();
      while (copied < min(total, kFirstCopies)) copy();
    }
  }
  // Tensor memory is taken after the kernel before has ended, which may hold some, and
  // before the kernel after may begin, which may want some.
  if (warp == 9) {
    grid_dependency_wait();
    take_tmem<PAIR>(&tmem_slot, 512);
  }
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the other block's barriers are there
  tc::fence_after_sync();
  allow_dependent_launch();
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
  if (warp >= 8) {
    if constexpr (!SWAP) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == 8) {
      if (lane == 0) {
        if constexpr (PAIR) grid_dependency_wait();
        uint32_t parity = 0;
        while (copied < total && !failed) {
          if (copied >= p.stages) {
            if (!wait(&empty[copy_st], parity, 90)) break;
            if (copy_st == p.stages - 1) parity ^= 1u;
          }
          copy();
        }
        // No arrival of the last instructions is on its way to a barrier here when the block ends, and so no copy is in
        // flight, which they waited for.  Those of a pair, which the first block issues, arrive in both blocks, and the
        // first block's own copy of one says nothing of the second block's.
        if (PAIR && rank != 0) tell(&others, &told, copied, 0);
        const OpenSteps open = open_steps(copied, p.stages);
        auto each_open = [&](auto one) {  // as long as it holds
          int st = open.stage;
          uint32_t phase = open.phase;
          bool ok = true;
          for (int step = open.from; ok && step < copied; ++step) {
            ok = one(st, phase);
            if (++st == p.stages) st = 0, phase ^= 1u;
          }
          return ok;
        };
        const bool ended = each_open([&](int st, uint32_t phase) { return wait(&empty[st], phase, 97); });
        if (PAIR && rank != 0 && !mbar_wait(&drain, 0, p.limit)) report(p.status, kDevTimeout, 98);
        // After a wait that ran out, the copies by themselves.  Both blocks' bytes of a pair count in the first one, which
        // may have stopped at an earlier step than the second one: it learns of the others (the second block may be at a
        // wait of its own first) and expects those bytes alone.
        if (!ended && (!PAIR || rank == 0)) {
          each_open([&](int st, uint32_t phase) { return mbar_wait(&full[st], phase, p.limit), true; });
          if (PAIR && mbar_wait(&told, 0, 2 * p.limit)) {
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
            for (int step = copied; step < others; ++step) {
              uint64_t* const bar = &full[step % p.stages];
              mbar_arrive_expect_tx(bar, p.stage_bytes);
              mbar_wait(bar, (uint32_t)(step / p.stages) & 1u, p.limit);
            }
          }
        }
      }
    } else if (warp == 9) {
      if (!PAIR || rank == 0) {
        const uint32_t at = smem_u32(ring);
        int st = 0, step = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int i = 0; i < my_tiles && ok; ++i) {
          for (int k = 0; k < ksteps; ++k, ++step) {
            const int acc = step % kAcc;
            ok = wait_warp(&full[st], parity, 92) && (step < kAcc || wait_warp(&acc_empty[acc], (uint32_t)(step / kAcc - 1) & 1u, 91));
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t ad = tc::smem_desc_sw128(at + st * p.stage_bytes);
            const uint64_t bd = tc::smem_desc_sw128(at + st * p.stage_bytes + kRowsA * kStep);
#pragma unroll
            for (int q = 0; q < 4; ++q)  // K = 32 is 32 bytes: 2 in the descriptors' address units
              mma_f8<PAIR>(tmem + acc * 2 * NC, ad + 2 * q, bd + 2 * q, p.idesc, q > 0);
            commit_one<PAIR>(&empty[st]);
            commit_one<PAIR>(&acc_full[acc]);
            if (++st == p.stages) st = 0, parity ^= 1u;
          }
        }
        // every instruction has finished before the block gives its tensor memory back
        commit_one<PAIR>(&drain);
        if (!mbar_wait(&drain, 0, p.limit)) report(p.status, kDevTimeout, 93);
      }
    } else if (warp == 10) {
      // scales, without waiting for them: a step's barrier counts the lanes whose copies have come
      grid_dependency_wait();
      const int64_t groups_b = sb.group == 1 ? sb.rows : (sb.rows + sb.group - 1) / sb.group;
      int ta = first / p.tiles_b, tb = first - ta * p.tiles_b, k = 0, st = 0;
      uint32_t parity = 1;
      for (int step = 0; step < total; ++step) {
        if (step >= kScaleRing && !wait_warp(&sc_empty[st], parity, 94)) break;
        float* const to = scales + st * kScales;
        const float* const pa = sa.scale + (kfirst + k) * sa.stride;
        const float* const pb = sb.scale + (kfirst + k) * sb.stride;
        const int64_t ra = (int64_t)ta * rows_a + rank_a;
        if (sa.group == 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) copy_scale(to + 32 * j + lane, pa + ra + 32 * j + lane, ra + 32 * j + lane < sa.rows);
        } else if (lane == 0) {
          copy_scale(to, pa + ra / kRowsA, true);
        }
        if constexpr (COLS) {
#pragma unroll
          for (int j = 0; j < 2 * NC / 32; ++j) {
            const int64_t r = (int64_t)tb * p.BN + 32 * j + lane;
            if (32 * j < p.BN) copy_scale(to + kRowsA + 32 * j + lane, pb + r, 32 * j + lane < p.BN && r < groups_b);
          }
        } else if (lane < 2) {  // a warpgroup's 128 columns have one
          const int64_t r = (int64_t)tb * (p.BN / kRowsA) + lane;
          copy_scale(to + kRowsA + lane, pb + r, r < groups_b);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sc_full[st])) : "memory");
        if (++st == kScaleRing) st = 0, parity ^= 1u;
        if (++k == ksteps) {
          k = 0;
          for (tb += stride; tb >= p.tiles_b; tb -= p.tiles_b) ++ta;
        }
      }
      // nor is one in flight when the block ends
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    if constexpr (!SWAP) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    grid_dependency_wait();
    const int wg = warp >> 2, quarter = warp & 3;  // the tensor-memory lanes a warp may read
    const int cb = wg * p.half, cols = min(p.half, p.BN - cb);
    const uint32_t from = tmem + cb + ((uint32_t)quarter << 21);
    int step = 0;
    bool ok = true;
    for (int i = 0; i < my_tiles && ok; ++i) {
      const int tile = first + i * stride, ta = tile / p.tiles_b, tb = tile - ta * p.tiles_b;
      const int64_t ra = (int64_t)ta * rows_a + rank_a + quarter * 32 + lane, rb = (int64_t)tb * p.BN + cb;
      F2 acc[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) acc[c] = 0;
      const float row_bias = SWAP && !shared && bias && ra < sa.rows ? load_one(bias, ra, p.dt) : 0.f;
      const int my_scale = sa.group == 1 ? quarter * 32 + lane : 0;
      uint32_t v[2][32];
      // 32 columns of a step's sums, from v[i], times its scales
      auto add = [&](int i, int c, int at_step) {
        const float* own = scales + at_step % kScaleRing * kScales;
        const float* w = own + kRowsA + (COLS ? cb + 32 * c : wg);
        const float scale = own[my_scale] * (COLS ? 1.f : *w);
        const F2 both = f2(scale, scale);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          float ws[4] = {};
          if (COLS) {
            const float4 four = *reinterpret_cast<const float4*>(w + j);
            ws[0] = four.x, ws[1] = four.y, ws[2] = four.z, ws[3] = four.w;
          }
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            F2& to = acc[16 * c + (j + e) / 2];
            const F2 value = f2(__uint_as_float(v[i][j + e]), __uint_as_float(v[i][j + e + 1]));
            to = COLS ? fma2(mul2(value, both), f2(ws[e], ws[e + 1]), to) : fma2(value, both, to);
          }
        }
      };
      auto begin = [&](int at_step) {  // until a step's sums and scales are there
        ok = wait_warp(&sc_full[at_step % kScaleRing], (uint32_t)(at_step / kScaleRing) & 1u, 95) &&
             wait_warp(&acc_full[at_step % kAcc], (uint32_t)(at_step / kAcc) & 1u, 96);
        tc::fence_after_sync();
        return from + at_step % kAcc * (2 * NC);
      };
      auto give_back = [&](int at_step) {  // all of the buffer has been read
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            arrive_at(peer_of(&acc_empty[at_step % kAcc], 0));
          else
            mbar_arrive(&acc_empty[at_step % kAcc]);
        }
      };
      auto used = [&](int at_step) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_empty[at_step % kScaleRing]);
      };
      if (SWAP && cols <= 32) {
        // two steps at a time: one's way from the barrier through tensor memory takes longer than its work
        for (int k = 0; k < ksteps; k += 2, step += 2) {
          const bool two = k + 1 < ksteps;
          const uint32_t at = begin(step);
          if (!ok) break;
          if (cols > 0) tmem_ld32(at, v[0]);
          if (two) {
            const uint32_t at1 = begin(step + 1);
            if (!ok) break;
            if (cols > 0) tmem_ld32(at1, v[1]);
          }
          tc::tmem_ld_wait();
          give_back(step);
          if (two) give_back(step + 1);
          if (cols > 0) add(0, 0, step);
          used(step);
          if (two) {
            if (cols > 0) add(1, 0, step + 1);
            used(step + 1);
          }
        }
        if (ksteps & 1) --step;
      } else {
        for (int k = 0; k < ksteps; ++k, ++step) {
          const uint32_t at = begin(step);
          if (!ok) break;
          // 32 columns at a time, two reads of tensor memory in flight: one's way takes some 200 cycles
          tmem_ld32(at, v[0]);
          tmem_ld32(at + 32, v[1]);
          tc::tmem_ld_wait();
          if (NC <= 64) give_back(step);
#pragma unroll
          for (int c = 0; c < NC / 32; c += 2) {
            add(0, c, step);
            if (c + 2 < NC / 32) tmem_ld32(at + 32 * (c + 2), v[0]);
            if (32 * (c + 1) < cols) add(1, c + 1, step);
            if (c + 3 < NC / 32) tmem_ld32(at + 32 * (c + 3), v[1]);
            if (c + 2 < NC / 32) tc::tmem_ld_wait();
            if (c + 4 >= NC / 32 && c + 2 < NC / 32) give_back(step);
          }
          used(step);
        }
      }
      if (!ok) {
        tc::tmem_ld_wait();
        break;
      }
      if constexpr (SWAP) {
        if (shared) {
          // this block's sums, [column][lane]; every copy into the ring has been read
          float* part = reinterpret_cast<float*>(ring) + quarter * 32 + lane + cb * kRowsA;
#pragma unroll
          for (int c = 0; c < NC; c += 16)
            if (c < cols) {
#pragma unroll
              for (int j = c; j < c + 16; ++j) part[j * kRowsA] = j & 1 ? hi(acc[j / 2]) : lo(acc[j / 2]);
            }
        } else if (ra < sa.rows) {
          const int rows = sb.rows - rb < cols ? (int)(sb.rows - rb) : cols;
#pragma unroll
          for (int c = 0; c < NC; c += 16)
            if (c < rows) {
#pragma unroll
              for (int j = c; j < c + 16; ++j)
                if (j < rows) store_one(y, (rb + j) * ys + ra, (j & 1 ? hi(acc[j / 2]) : lo(acc[j / 2])) + row_bias, p.dt);
            }
        }
      } else {
        const int es = p.dt == kF32 ? 4 : 2, per = 128 / es;  // columns in 128 bytes
        unsigned char* const mine = out + warp * kOutBytes;
        const int64_t r0 = (int64_t)ta * rows_a + rank_a + quarter * 32;
        if (bias) {
          const int c = wg * NC + quarter * 32 + lane;
          const int64_t r = (int64_t)tb * p.BN + c;
          col_bias[c] = r < sb.rows ? load_one(bias, r, p.dt) : 0.f;
          bar_sync(1 + wg, 128);
#pragma unroll
          for (int k = 0; k < NC / 4; ++k) {
            const float4 add = reinterpret_cast<const float4*>(col_bias + wg * NC)[k];
            acc[2 * k] = add2(acc[2 * k], f2(add.x, add.y)), acc[2 * k + 1] = add2(acc[2 * k + 1], f2(add.z, add.w));
          }
          bar_sync(1 + wg, 128);
        }
        // 32 rows x 128 bytes a piece, 16 bytes k of row r at k ^ (r % 8), as TMA has them
#pragma unroll
        for (int h = 0; h < NC / 32; ++h) {  // 32 columns: a piece of fp32, half a piece else
          const int piece = es == 4 ? h & 1 : h >> 1;
          unsigned char* const to = mine + piece * 4096 + lane * 128;
          if (es == 4 ? (h & 1) == 0 : h == 0) {  // the pieces of the stores before have been read
            if (lane == 0) tma_store_wait_read();
            __syncwarp();
          }
          if (es == 4) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(to + ((k ^ (lane & 7)) << 4)) =
                  make_float4(lo(acc[16 * h + 2 * k]), hi(acc[16 * h + 2 * k]), lo(acc[16 * h + 2 * k + 1]), hi(acc[16 * h + 2 * k + 1]));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float v0 = lo(acc[16 * h + 4 * k + e]), v1 = hi(acc[16 * h + 4 * k + e]);
                w[e] = p.dt == kF16 ? round_pair<__half>(v0, v1) : round_pair<__nv_bfloat16>(v0, v1);
              }
              *reinterpret_cast<uint4*>(to + (((4 * (h & 1) + k) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if ((h & 1) == 0) continue;
          }
          const int64_t col = rb + (es == 4 ? 32 * h : 32 * (h - 1));
          if (p.y_map) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && r0 < sa.rows && col < sb.rows) {
              store_2d(&ymap, mine + piece * 4096, (int)col, (int)r0);
              tma_store_commit();
            }
          } else {  // rows of y off 16 bytes
            __syncwarp();
            const int room = sb.rows - col < per ? (int)(sb.rows - col) : per;  // columns that y has
            for (int row = 0; row < 32 && r0 + row < sa.rows; ++row)
              for (int c = lane; c < room; c += 32) {
                const unsigned char* at = mine + piece * 4096 + row * 128 + (((c * es >> 4) ^ (row & 7)) << 4) + (c * es & 15);
                if (es == 4)
                  static_cast<float*>(y)[(r0 + row) * ys + col + c] = *reinterpret_cast<const float*>(at);
                else
                  static_cast<uint16_t*>(y)[(r0 + row) * ys + col + c] = *reinterpret_cast<const uint16_t*>(at);
              }
            __syncwarp();
          }
        }
      }
    }
    if (PAIR && lane == 0) tma_store_wait_all();
  }
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // no block leaves or gives its tensor memory back while the other works
  if (warp == 9) {
    tc::fence_after_sync();
    return_tmem<PAIR>(tmem, 512);
  }
  if constexpr (SWAP) {
    if (shared) {
      const int ta = first / p.tiles_b, tb = first - ta * p.tiles_b;
      const int64_t n = (int64_t)ta * kRowsA + 4 * lane, m0 = (int64_t)tb * p.BN;  // a warp takes whole rows of y
      const int rows = sb.rows - m0 < p.BN ? (int)(sb.rows - m0) : p.BN;
      float add[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) add[e] = bias && n + e < sa.rows ? load_one(bias, n + e, p.dt) : 0.f;
      const uint32_t part = smem_u32(ring) + (uint32_t)lane * 16u;
      cluster_sync();  // every block's sums are there
      for (int c = rank + warp * p.split; c < rows; c += kF8Threads / 32 * p.split) {
        float o[4] = {};
        for (int k = 0; k < p.split; ++k) {
          const float4 v = ld_cluster(part + (uint32_t)c * (kRowsA * 4), k);
          o[0] += v.x, o[1] += v.y, o[2] += v.z, o[3] += v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < sa.rows) store_one(y, (m0 + c) * ys + n + e, o[e] + add[e], p.dt);
      }
      cluster_sync();  // no block leaves while another reads its sums
    }
  }
}

uint32_t idesc_f8(bool ae5, bool be5, int M, int N) {
  return (1u << 4) | ((ae5 ? 1u : 0u) << 7) | ((be5 ? 1u : 0u) << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Blocks of clusters of `split` that run at once, one an SM: with 152 SMs the device
// reports 152 of 2, 138 of 3, 144 of 4, 140 of 5, 138 of 6, 105 of 7 and 120 of 8.
int share_sms(int split, int sms) { return split <= 2 ? sms : split <= 6 ? sms * 9 / 10 : sms * 3 / 4; }

// Dynamic shared memory: alignment, ring, rows of y on their way out, scales, bias.
size_t f8_smem(bool swap, bool cols, const F8Plan& p) {
  const int columns = swap ? 128 : 256;
  return 1024 + (size_t)p.stages * p.stage_bytes + kScaleRing * (kRowsA + (cols ? columns : 4)) * 4 +
         (swap ? 0 : 8 * kOutBytes + columns * 4);
}

// The form and its tile, by the time that the steps of the busiest block take.  A step of K = 128 took, ns: SWAP
// with 16 ... 48 columns 300 (its way through the warps), 64: 370, 96: 460, 128: 500; pairs 520.  Sharing a tile costs
// the sums' way through the blocks' shared memory.  In a graph, us: 16 x 8192 x 2048 8.2, 64 x 8192 x 2048 9.9,
// 197 x 5000 x 2048 11.1 (three tiles of 80; in pairs 13.6), 256 x 4864 x 2048 10.5, 128 x 8192 x 8192 21.8 (two blocks a
// tile), 1 x 4096 x 4096 7.8 (four).
bool f8_plan(const MatmulF8Args& m, const DeviceInfo& dev, F8Plan* p, bool* swap) {
  const int steps = (m.K + kStep - 1) / kStep;
  int64_t best = -1;
  const int64_t tiles_n = (m.N + kRowsA - 1) / kRowsA;
  for (int bn = 16; bn <= 128; bn += 16) {
    if (bn > 16 && m.M <= bn - 16) break;
    const int64_t tiles_m = (m.M + bn - 1) / bn, tiles = tiles_m * tiles_n, rounds = (tiles + dev.num_sms - 1) / dev.num_sms;
    if (tiles > 0x7fffffff) continue;
    for (int split = 1; split <= std::min(kMaxSplit, steps); ++split) {
      if (split > 1 && (split == 7 || tiles * split > share_sms(split, dev.num_sms))) continue;
      const int per = (steps + split - 1) / split;
      if (split > 1 && per * (split - 1) >= steps) continue;
      const int64_t cost = rounds * per * std::max(300, 180 + 3 * bn) + (split > 1 ? 1500 + 10 * bn : 0);
      if (best < 0 || cost < best) {
        best = cost;
        *swap = true;
        p->BN = bn, p->tiles_b = (int)tiles_m, p->tiles = (int)tiles, p->split = split, p->per = per;
      }
    }
  }
  const int64_t pair_tiles = ((m.M + 255) / 256) * ((m.N + 255) / 256);
  if (pair_tiles <= 0x7fffffff && dev.num_sms >= 2) {
    const int64_t cost = (pair_tiles + dev.num_sms / 2 - 1) / (dev.num_sms / 2) * (steps * 520 + 1300);
    if (best < 0 || cost < best) {
      best = cost;
      *swap = false;
      p->BN = 256, p->tiles_b = (m.N + 255) / 256, p->tiles = (int)pair_tiles, p->split = 1, p->per = steps;
    }
  }
  if (best < 0) return false;
  p->ksteps = steps;
  if ((int64_t)(p->tiles / std::max(1, dev.num_sms / 2) + 1) * steps > 0x7fffffff) return false;
  p->half = *swap ? (p->BN / 16 + 1) / 2 * 16 : 128;
  p->stage_bytes = (uint32_t)(kRowsA + (*swap ? p->BN : kRowsA)) * kStep;
  p->idesc = *swap ? idesc_f8(m.we5, m.xe5, kRowsA, p->BN) : idesc_f8(m.xe5, m.we5, 2 * kRowsA, p->BN);
  p->stages = 0;
  const int rest = (int)f8_smem(*swap, *swap || m.w_rows == 1, *p);
  p->stages = std::min(kMaxStages, (dev.max_smem_optin - 1024 - rest) / (int)p->stage_bytes);  // barriers: below 1 KB
  return p->stages >= 2;
}

bool byte_map(CUtensorMap* map, const uint8_t* p, int64_t rows, int K, int64_t pitch, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)K, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)pitch};
  const uint32_t box[2] = {kStep, (uint32_t)box_rows}, ones[2] = {1, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, dims, strides, box, ones, CU_TENSOR_MAP_SWIZZLE_128B) ==
         CUDA_SUCCESS;
}

// Rows of y as the pair form stores them: 32 rows x 128 bytes.  A store writes whole 16 bytes, with zeros past the last
// column of a row that ends inside them, so that rows end on 16 bytes, too.
bool y_map(CUtensorMap* map, const MatmulF8Args& m, DType dt) {
  const int es = dtype_bytes(dt);
  if ((m.ys * es & 15) || ((int64_t)m.N * es & 15) || (reinterpret_cast<uintptr_t>(m.y) & 15)) return false;
  const uint64_t dims[2] = {(uint64_t)m.N, (uint64_t)m.M};
  const uint64_t strides[1] = {(uint64_t)m.ys * es};
  const uint32_t box[2] = {(uint32_t)(128 / es), 32}, ones[2] = {1, 1};
  const CUtensorMapDataType type = dt == kF32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dt == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return encode_tiled(map, type, 2, m.y, dims, strides, box, ones, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}

template <bool SWAP, bool COLS>
cudaError_t launch(const MatmulF8Args& m, F8Plan p, const LaunchArgs& a, const DeviceInfo& dev) {
  CUtensorMap amap = {}, bmap = {}, out = {};
  if (!(SWAP ? byte_map(&amap, m.wq, m.N, m.K, m.wp, kRowsA) && byte_map(&bmap, m.xq, m.M, m.K, m.xp, p.BN)
             : byte_map(&amap, m.xq, m.M, m.K, m.xp, kRowsA) && byte_map(&bmap, m.wq, m.N, m.K, m.wp, kRowsA)))
    return cudaErrorInvalidValue;
  p.y_map = !SWAP && y_map(&out, m, a.dt);
  const size_t smem = f8_smem(SWAP, COLS, p);
  static SmemAttr most;
  const cudaError_t e = most.ensure(mmf8_kernel<SWAP, COLS>, dev.device, (int)smem);
  if (e != cudaSuccess) return e;
  const Side x = {m.sx, m.xss, m.M, 1}, w = {m.sw, m.wss, m.N, m.w_rows};
  const int cluster = SWAP ? p.split : 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cluster > 1 && SWAP ? p.tiles * cluster : std::min(p.tiles, dev.num_sms / cluster) * cluster));
  cfg.blockDim = dim3(kF8Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, mmf8_kernel<SWAP, COLS>, amap, bmap, out, SWAP ? w : x, SWAP ? x : w, m.y, m.bias, m.ys, p);
}

}  // namespace

cudaError_t matmul_f8_launch(const MatmulF8Args& m, const LaunchArgs& a, const DeviceInfo& dev) {
  F8Plan p = {};
  bool swap = false;
  if (!f8_plan(m, dev, &p, &swap)) return cudaErrorInvalidConfiguration;  // more tiles than 31 bits count
  p.dt = a.dt, p.status = a.status, p.limit = a.wait_limit_ns;
  if (swap) return launch<true, true>(m, p, a, dev);
  return m.w_rows == 1 ? launch<false, true>(m, p, a, dev) : launch<false, false>(m, p, a, dev);
}

}  // namespace gconv
