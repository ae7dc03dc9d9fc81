// Matrix product in 8-bit floating point with a scale for each block of 128:
//
//   C[m, n] = sum_kb sa[kb, m] sb[n / 128, kb] sum_{k in block kb} A[m, k] B[n, k]  (+ bias[n])
//
// A [M, K] and B [N, K] are e4m3, sa one fp32 scale per row and 128 channels,
// sb one per 128 x 128 block; C is bf16 or fp32.  The inner sums run on the
// tensor cores (tcgen05, kind::f8f6f4, fp32 accumulation); each block's sum
// leaves tensor memory once and is scaled and added into fp32 registers.
//
// Two CTAs on neighbouring SMs (a cluster) work on one 256 x 256 tile (256 x 128
// where there are few): each brings its 128 rows of A and half of B's rows, and
// one instruction multiplies on both (cta_group::2).  So an SM takes in 32 KB
// per k block instead of the 48 KB that a 128 x 256 tile of its own would need.
//
// Pairs stay and walk the tiles.  In each CTA a producer thread brings one
// 128-byte-wide k block of A and B per step into a ring of shared-memory stages
// by TMA (K tails and edge rows are filled with zeros, which add nothing), and
// two warps bring the products of the scales.  An issuer thread in the pair's
// first CTA multiplies a stage into one of two tensor-memory buffers; in both
// CTAs two warpgroups, each with half the columns, add buffer after buffer into
// their registers while the next block is multiplied.  Results leave through
// shared memory and TMA stores, which drop what lies past M and N.
//
// Measured, 75,600 x 5,120 x 15,360: 6.0 to 6.8 ms in short runs, 7.0 to 7.2 ms in
// long ones (1.98 to 1.66 PFLOP/s).  What bounds it first is the adding warps'
// chain per block -- wait, load, add: with zeros as data, which stay below the
// power limit, 5.1 to 5.7 ms between GPUs, 1,040 to 1,160 cycles a block at 512 of
// tensor work.  With normal data the power limit comes on top (long runs are at
// 1.6 GHz); the multiplications and loads alone took 4.8 ms, 3.6 with zeros.  So the
// chain is kept short: a stage's one barrier says that it is free, that its sums
// are there and that the scales are, and the load of the next 32 columns, of the
// next block too, is under way while 32 are added.
#include "layer_common.cuh"
#include "kernels.h"
#undef VEDA_SRC_ID
#define VEDA_SRC_ID 11   // bounds-check site id of this file (debug builds)

namespace veda {
// Instruction descriptor, kind::f8f6f4: e4m3 A/B (format 0), fp32 D, both K-major.
__host__ __device__ constexpr uint32_t make_idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address in the cluster of this CTA's shared address, seen in the CTA of `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// A consumer warp has read a block's sums and scales: its first lane arrives at
// the buffer's barrier in the first CTA and at the scales' barrier in its own.
// No branch around them, and no arrival left out where one of four would do: a
// test of the block's number cost 2% at 75,600 x 5,120 x 15,360, this 0.5%.  No release at cluster scope either, which waits for the
// thread's memory traffic (a microsecond per block): all that the first arrival
// has to order are tensor-memory reads, by tcgen05.fence before it.
__device__ __forceinline__ void arrive_read(bool first, uint32_t sums_cluster_addr, uint32_t scales_bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%1];\n\t}" ::"r"(sums_cluster_addr),
      "r"(scales_bar), "r"((int)first)
      : "memory");
}

// The pair's forms (cta_group::2) of what veda_common.cuh has for one CTA.
namespace pair {
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Into this CTA's shared memory, completion counted at a barrier of either CTA.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 operands, fp32 accumulate, K = 32, over both CTAs.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives at the barrier of this address in both CTAs once the multiplications so far are done.
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
}  // namespace pair

// Shared memory of the kernel for 256 x BN tiles.
template <int BN>
struct GemmCfg {
  static constexpr int kThreads = 384;
  static constexpr int kStages = 4;
  static constexpr int kBuffers = 512 / BN;           // of tensor memory
  static constexpr int kA = 128 * 128, kB = BN / 2 * 128;   // a CTA's part of A and of B per stage
  static constexpr int kOffB = kStages * kA;
  static constexpr int kOffOut = kOffB + kStages * kB;      // per consumer warp two pieces of 32 rows x 128 bytes
  static constexpr int kOffScale = kOffOut + 8 * 2 * 4096;  // [8 slots][column half][row]
  static constexpr int kOffBar = kOffScale + 8 * 256 * 4;
  static constexpr int kOffMisc = kOffBar + 16 * 8;
  static constexpr size_t kSmem = 1024 + kOffMisc + 64;
};

enum {
  GBAR_FULL = 0,    // +stage (4): both CTAs' operands have come (the first CTA's barrier counts)
  GBAR_DONE = 4,    // +stage (4): its multiplications are done: the stage is free, the sums are there; and so are
                    // the products of this CTA's scales, from the warps that write them
  GBAR_DFREE = 8,   // +buffer (2 or 4): both CTAs' consumers have read it (the first CTA's barrier counts)
  GBAR_SFREE = 12,  // +half of the scales' slots (2): this CTA's consumers have read those of four blocks
};

__device__ __forceinline__ bool gemm_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, timeout_ns));
}

// The limit of the waits for copies and multiplications already in flight after
// another wait ran out: they take microseconds, whatever limit the caller set.
__device__ __forceinline__ uint64_t drain_limit(uint64_t timeout_ns) {
  return timeout_ns > 50000000ull ? timeout_ns : 50000000ull;
}

// Waits for the tensor-memory loads in flight, among them the one into v: what
// follows reads v from here, not from the load.
__device__ __forceinline__ void tmem_ld_wait32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld_wait16(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}

// Tile t in an order that keeps a wave's operands in L2: groups of 8 tile rows,
// column by column inside a group.
__device__ __forceinline__ void gemm_tile(const GemmArgs& A, int t, int* m, int* n) {
  const int per_group = 8 * A.tiles_n;
  const int first = t / per_group * 8, r = t % per_group;
  const int rows = min(8, A.tiles_m - first);
  *m = first + r % rows;
  *n = r / rows;
}

template <int BN, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(384, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmC, const __grid_constant__ GemmArgs A) {
  using C = GemmCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sA = smem_u32(smem), sB = smem_u32(smem + C::kOffB), bar0 = smem_u32(smem + C::kOffBar);
  auto bar = [&](int b) { return bar0 + 8u * (uint32_t)b; };
  int* misc = reinterpret_cast<int*>(smem + C::kOffMisc);   // [0] tmem base, [1] abort
  volatile int* abort = misc + 1;
  const uint64_t tmo = A.timeout_ns;
  const int rank = (int)cluster_rank(), first_tile = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (tid == 0) {
    misc[1] = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(GBAR_FULL + s), 1);
      mbar_init(bar(GBAR_DONE + s), 3);
    }
    for (int s = 0; s < C::kBuffers; ++s) mbar_init(bar(GBAR_DFREE + s), 16);
    for (int s = 0; s < 2; ++s) mbar_init(bar(GBAR_SFREE + s), 4 * 8);
    fence_mbar_init();
  }
  if (warp == 1) pair::tmem_alloc(smem_u32(&misc[0]), 512);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      int it = 0;
      bool ok = true;
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmB);
      tma_prefetch_desc(&tmC);
      const uint32_t full0 = map_rank(bar(GBAR_FULL), 0);
      for (int t = first_tile; ok && t < A.tiles; t += pairs) {
        int m, n;
        gemm_tile(A, t, &m, &n);
        const int row = m * 256 + rank * 128, col = n * BN + rank * (BN / 2);
        for (int kb = 0; kb < A.kblocks; ++kb, ++it) {
          const int st = it % C::kStages, fill = it / C::kStages;
          if (fill >= 1 && !(ok = mbar_wait(bar(GBAR_DONE + st), (fill - 1) & 1, abort, tmo))) break;
          if (VEDA_IN_BOUNDS(m * 256 < A.M && n * BN < A.N && kb * 128 < A.K)) {
            if (rank == 0) mbar_arrive_expect_tx(bar(GBAR_FULL + st), 2 * (C::kA + C::kB));
            pair::tma_load_2d(sA + st * C::kA, &tmA, full0 + 8 * st, kb * 128, row);
            pair::tma_load_2d(sB + st * C::kB, &tmB, full0 + 8 * st, kb * 128, col);
          }
        }
      }
      // The last fills: on a failure the copies in flight are waited for (at
      // the barriers that count them); otherwise the signals that they were
      // used, the last things to come to this CTA's barriers from outside.
      int dummy = 0;
      const bool failed = *abort != 0;
      for (int i = it > C::kStages ? it - C::kStages : 0; i < it && !(failed && rank); ++i)
        mbar_wait(bar((failed ? GBAR_FULL : GBAR_DONE) + i % C::kStages), (i / C::kStages) & 1, &dummy, drain_limit(tmo));
    } else if (warp == 1 && lane == 0 && rank == 0) {
      constexpr uint32_t idesc = make_idesc_e4m3(256, BN);
      const uint64_t da0 = make_sdesc_sw128(sA, 16, 1024), db0 = make_sdesc_sw128(sB, 16, 1024);
      int it = 0;
      bool ok = true;
      for (int t = first_tile; ok && t < A.tiles; t += pairs) {
        for (int kb = 0; kb < A.kblocks; ++kb, ++it) {
          const int st = it % C::kStages, buf = it % C::kBuffers;
          if (!(ok = mbar_wait(bar(GBAR_FULL + st), (it / C::kStages) & 1, abort, tmo))) break;
          if (it >= C::kBuffers && !(ok = mbar_wait(bar(GBAR_DFREE + buf), (it / C::kBuffers - 1) & 1, abort, tmo))) break;
          tc_fence_after();
          const uint64_t da = da0 + (uint64_t)((st * C::kA) >> 4), db = db0 + (uint64_t)((st * C::kB) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            pair::umma_f8(tmem + buf * BN, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
          pair::umma_commit(bar(GBAR_DONE + st));
        }
      }
      // The consumers have seen the last commit, or a wait ran out; then the
      // multiplications in flight are waited for here, again with a limit.
      if (!ok && it > 0) {
        int dummy = 0;
        mbar_wait(bar(GBAR_DONE + (it - 1) % C::kStages), ((it - 1) / C::kStages) & 1, &dummy, drain_limit(tmo));
      }
    } else if (warp >= 2) {
      // The products sa sb, one warp per column half, two k blocks at a time.
      // They are written, read and freed inside a CTA, at barriers of its own
      // (what one CTA's threads do is not ordered for the other's by a signal
      // through the issuer).  Block it has slot it & 7; four slots are free
      // again when the consumers have read all four.
      const int half = warp - 2;
      float* dst = reinterpret_cast<float*>(smem + C::kOffScale) + half * 128 + lane;
      int it = 0;
      bool ok = true;
      for (int t = first_tile; ok && t < A.tiles; t += pairs) {
        int m, n;
        gemm_tile(A, t, &m, &n);
        const int row = m * 256 + rank * 128 + lane;
        const float* pb = A.sb + (long long)min(BN == 256 ? n * 2 + half : n, A.nblocks - 1) * A.kblocks;
        float next[2][4], nb[2];
        auto fetch = [&](int kb) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int k = min(kb + j, A.kblocks - 1);
            nb[j] = __ldg(pb + k);
#pragma unroll
            for (int r = 0; r < 4; ++r) next[j][r] = __ldg(A.sa + ((long long)k * A.M + min(row + r * 32, A.M - 1)));
          }
        };
        fetch(0);
        for (int kb = 0; ok && kb < A.kblocks; kb += 2) {
          float v[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[j][r] = next[j][r] * nb[j];
          }
          if (kb + 2 < A.kblocks) fetch(kb + 2);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (kb + j >= A.kblocks) break;
            const int st = it % C::kStages, fill = it / C::kStages, turn = it >> 3;
            if ((it & 3) == 0 && turn >= 1 &&
                !(ok = gemm_wait(bar(GBAR_SFREE + ((it >> 2) & 1)), (turn - 1) & 1, abort, tmo)))
              break;
            // This block's phase of its stage has begun.
            if (fill >= 1 && !(ok = gemm_wait(bar(GBAR_DONE + st), (fill - 1) & 1, abort, tmo))) break;
#pragma unroll
            for (int r = 0; r < 4; ++r) dst[(it & 7) * 256 + r * 32] = v[j][r];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(GBAR_DONE + st));
            ++it;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    constexpr int HN = BN / 2;               // columns of this warpgroup
    constexpr int PC = 128 / sizeof(TO);     // columns of an output piece
    const int half = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * HN);
    const uint32_t free0 = map_rank(bar(GBAR_DFREE), 0);
    uint8_t* out = smem + C::kOffOut + (warp - 4) * 8192;
    const float* scales = reinterpret_cast<const float*>(smem + C::kOffScale) + half * 128 + quarter * 32 + lane;
    int it = 0, pieces = 0;
    bool ok = true;
    for (int t = first_tile; ok && t < A.tiles; t += pairs) {
      // One stream of 32-column pieces through all blocks: while a piece is
      // added, the next one -- of the next block too -- is on its way.
      uint64_t acc[HN / 2];
#pragma unroll
      for (int j = 0; j < HN / 2; ++j) acc[j] = 0;
      float v[2][32];
      float sc = 0.f, nsc = 0.f;
      if (!(ok = gemm_wait(bar(GBAR_DONE + it % C::kStages), (it / C::kStages) & 1, abort, tmo))) break;
      tc_fence_after();
      sc = scales[(it & 7) * 256];
      tmem_ld32(t_lane + it % C::kBuffers * BN, v[0]);
      for (int kb = 0; kb < A.kblocks; ++kb, ++it) {
        const uint32_t from = t_lane + it % C::kBuffers * BN;
#pragma unroll
        for (int c = 0; c < HN / 32; ++c) {
          tmem_ld_wait32(v[c & 1]);
          if (c + 1 < HN / 32) {
            tmem_ld32(from + (c + 1) * 32, v[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            arrive_read(lane == 0, free0 + 8u * (uint32_t)(it % C::kBuffers), bar(GBAR_SFREE + ((it >> 2) & 1)));
            if (kb + 1 < A.kblocks) {
              const int next = it + 1;
              ok = gemm_wait(bar(GBAR_DONE + next % C::kStages), (next / C::kStages) & 1, abort, tmo);
              if (ok) {
                tc_fence_after();
                nsc = scales[(next & 7) * 256];
                tmem_ld32(t_lane + next % C::kBuffers * BN, v[0]);
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[c * 16 + j] = f2_fma(f2(v[c & 1][2 * j], v[c & 1][2 * j + 1]), f2_all(sc), acc[c * 16 + j]);
        }
        if (!ok) break;
        sc = nsc;
      }
      int m, n;
      gemm_tile(A, t, &m, &n);
      const int row0 = m * 256 + rank * 128 + quarter * 32, col0 = n * BN + half * HN;
      if (!ok || row0 >= A.M) continue;
#pragma unroll
      for (int p = 0; p < HN / PC; ++p) {
        const int col = col0 + p * PC;
        if (col >= A.N) break;
        uint8_t* piece = out + (pieces++ & 1) * 4096;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");   // the piece before last has left
        __syncwarp();
#pragma unroll
        for (int u = 0; u < PC / 8; ++u) {     // 8 columns at a time
          uint64_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = acc[(p * PC + 8 * u) / 2 + k];
          if (A.bias != nullptr && col + 8 * u < A.N) {
            uint64_t b[4];
            load_pairs(A.bias + col + 8 * u, b);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = f2_add(v[k], b[k]);
          }
          const Words<TO> w = to_words<TO>(v);
#pragma unroll
          for (int k = 0; k < (int)(sizeof(TO) / 2); ++k) {
            const int unit = u * (int)(sizeof(TO) / 2) + k;
            *reinterpret_cast<uint4*>(piece + lane * 128 + ((unit ^ (lane & 7)) << 4)) = w.u[k];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (VEDA_IN_BOUNDS(row0 < A.M && col < A.N))
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                             reinterpret_cast<uint64_t>(&tmC)),
                         "r"(smem_u32(piece)), "r"(col), "r"(row0)
                         : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();   // nobody leaves while the other may still signal its barriers or read its operands
  if (warp == 1) {
    tc_fence_after();
    pair::tmem_dealloc(tmem, 512);
  }
}

// ---- few rows ----
//
// With few tiles the weights' bytes are the work, and they should come through
// as many SMs as there are.  So the roles change: 128 rows of the weights are
// the tensor core's M, and TN = 16, 32 or 64 rows of A its N; and a cluster of
// up to 8 CTAs shares a tile's k blocks.  Each CTA adds its blocks up in
// registers as above (a thread has one weight row and TN sums); the partial
// sums go to shared memory, and each CTA adds all of them, in rank order, for
// its share of A's rows.  Two CTAs fit an SM, with some 100 KB of operands in
// flight each.
template <int TN>
struct FewCfg {
  static constexpr int kThreads = 256;
  static constexpr int kStages = TN == 16 ? 6 : TN == 32 ? 5 : 4;
  static constexpr int kBuffers = 4;
  static constexpr int kSlots = 16;        // of scales: at least stages + buffers
  static constexpr int kW = 128 * 128, kX = TN * 128;
  static constexpr int kOffX = kStages * kW;
  static constexpr int kOffScale = kOffX + kStages * kX;
  static constexpr int kOffBar = kOffScale + kSlots * TN * 4;
  static constexpr int kOffMisc = kOffBar + 16 * 8;
  static constexpr size_t kSmem = 1024 + kOffMisc + 64;
  static constexpr uint32_t kTmemCols = kBuffers * TN;
  static_assert(TN * 128 * 4 <= kOffX && kSlots >= kStages + kBuffers, "partial sums and scales fit");
};

enum {
  FBAR_FULL = 0,    // +stage (6): operands and scales have come
  FBAR_DONE = 6,    // +stage (6): its multiplications are done
  FBAR_DFREE = 12,  // +buffer (4)
};

// D[tmem] (+)= A[smem] * B[smem]^T in one CTA, e4m3 operands, fp32 accumulate, K = 32.
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int TN, typename TO>
__global__ void __launch_bounds__(256, 2)
    gemm_few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ GemmArgs A) {
  using C = FewCfg<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sW = smem_u32(smem), sX = smem_u32(smem + C::kOffX), bar0 = smem_u32(smem + C::kOffBar);
  auto bar = [&](int b) { return bar0 + 8u * (uint32_t)b; };
  float* scales = reinterpret_cast<float*>(smem + C::kOffScale);   // [slot][TN]
  int* misc = reinterpret_cast<int*>(smem + C::kOffMisc);          // [0] tmem base, [1] abort
  volatile int* abort = misc + 1;
  const uint64_t tmo = A.timeout_ns;
  const int rank = (int)cluster_rank(), tile = blockIdx.x / A.split;
  const int n0 = tile % A.tiles_n * 128, m0 = tile / A.tiles_n * TN;
  const int kb0 = (int)((long long)A.kblocks * rank / A.split), kb1 = (int)((long long)A.kblocks * (rank + 1) / A.split);
  const int count = kb1 - kb0;

  if (tid == 0) {
    misc[1] = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(FBAR_FULL + s), 2);
      mbar_init(bar(FBAR_DONE + s), 1);
    }
    for (int s = 0; s < C::kBuffers; ++s) mbar_init(bar(FBAR_DFREE + s), 4);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&misc[0]), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    int it = 0;
    for (; it < count; ++it) {
      const int st = it % C::kStages, fill = it / C::kStages;
      if (fill >= 1 && !mbar_wait(bar(FBAR_DONE + st), (fill - 1) & 1, abort, tmo)) break;
      if (VEDA_IN_BOUNDS(n0 < A.N && m0 < A.M && (kb0 + it) * 128 < A.K)) {
        mbar_arrive_expect_tx(bar(FBAR_FULL + st), C::kW + C::kX);
        tma_load_2d(sW + st * C::kW, &tmW, bar(FBAR_FULL + st), (kb0 + it) * 128, n0);
        tma_load_2d(sX + st * C::kX, &tmX, bar(FBAR_FULL + st), (kb0 + it) * 128, m0);
      }
    }
    if (*abort) {
      int dummy = 0;
      for (int i = it > C::kStages ? it - C::kStages : 0; i < it; ++i)
        mbar_wait(bar(FBAR_FULL + i % C::kStages), (i / C::kStages) & 1, &dummy, drain_limit(tmo));
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = make_idesc_e4m3(128, TN);
    const uint64_t dw0 = make_sdesc_sw128(sW, 16, 1024), dx0 = make_sdesc_sw128(sX, 16, 1024);
    int it = 0;
    for (; it < count; ++it) {
      const int st = it % C::kStages, buf = it % C::kBuffers;
      if (!mbar_wait(bar(FBAR_FULL + st), (it / C::kStages) & 1, abort, tmo)) break;
      if (it >= C::kBuffers && !mbar_wait(bar(FBAR_DFREE + buf), (it / C::kBuffers - 1) & 1, abort, tmo)) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_f8_ss(tmem + buf * TN, dw0 + (uint64_t)((st * C::kW) >> 4) + 2 * kk,
                   dx0 + (uint64_t)((st * C::kX) >> 4) + 2 * kk, idesc, kk > 0 ? 1u : 0u);
      umma_commit(bar(FBAR_DONE + st));
    }
    if (it > 0) {   // the last multiplications, also after a wait ran out
      int dummy = 0;
      mbar_wait(bar(FBAR_DONE + (it - 1) % C::kStages), ((it - 1) / C::kStages) & 1, &dummy, drain_limit(tmo));
    }
  } else if (warp == 2) {
    // The products sa sb of TN rows, two blocks ahead in registers.  A slot is
    // written again 16 blocks later: the stage's block before has been
    // multiplied then, so the buffer of the fourth before that was free, so its
    // scales, and all before, have been read.
    constexpr int R = TN > 32 ? 2 : 1;
    const float* pb = A.sb + (long long)(n0 / 128) * A.kblocks;
    const float* pa[R];
    float next[2][R], nb[2];
#pragma unroll
    for (int r = 0; r < R; ++r) pa[r] = A.sa + min(m0 + r * 32 + lane, A.M - 1);
    auto fetch = [&](int it) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = min(kb0 + it + j, A.kblocks - 1);
        nb[j] = __ldg(pb + k);
#pragma unroll
        for (int r = 0; r < R; ++r) next[j][r] = __ldg(pa[r] + (long long)k * A.M);
      }
    };
    fetch(0);
    bool ok = true;
    for (int i = 0; ok && i < count; i += 2) {
      float v[2][R];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int r = 0; r < R; ++r) v[j][r] = next[j][r] * nb[j];
      }
      if (i + 2 < count) fetch(i + 2);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int it = i + j, st = it % C::kStages, fill = it / C::kStages;
        if (it >= count) break;
        if (fill >= 1 && !(ok = gemm_wait(bar(FBAR_DONE + st), (fill - 1) & 1, abort, tmo))) break;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r * 32 + lane < TN) scales[(it % C::kSlots) * TN + r * 32 + lane] = v[j][r];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(FBAR_FULL + st));
      }
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    float acc[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[j] = 0.f;
    for (int it = 0; it < count; ++it) {
      const int st = it % C::kStages, buf = it % C::kBuffers;
      if (!gemm_wait(bar(FBAR_DONE + st), (it / C::kStages) & 1, abort, tmo)) break;
      tc_fence_after();
      float v[TN], sc[TN];
      if constexpr (TN == 16) {
        tmem_ld16(t_lane + buf * TN, v);
      } else {
#pragma unroll
        for (int c = 0; c < TN; c += 32) tmem_ld32(t_lane + buf * TN + c, v + c);
      }
      const float4* s4 = reinterpret_cast<const float4*>(scales + (it % C::kSlots) * TN);
#pragma unroll
      for (int j = 0; j < TN / 4; ++j) {
        const float4 s = s4[j];
        sc[4 * j] = s.x, sc[4 * j + 1] = s.y, sc[4 * j + 2] = s.z, sc[4 * j + 3] = s.w;
      }
      if constexpr (TN == 16) {
        tmem_ld_wait16(v);
      } else {
#pragma unroll
        for (int c = 0; c < TN; c += 32) tmem_ld_wait32(v + c);
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[j] = fmaf(v[j], sc[j], acc[j]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(FBAR_DFREE + buf));
    }
    // All operands have been multiplied, so their room is free.
    float* part = reinterpret_cast<float*>(smem);   // [TN][128]
#pragma unroll
    for (int j = 0; j < TN; ++j) part[j * 128 + row] = acc[j];
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  const int row = tid & 127, n = n0 + row;
  TO* out = static_cast<TO*>(A.out);
  const int t0 = TN * rank / A.split, t1 = TN * (rank + 1) / A.split;
  if (n < A.N) {
    const float bias = A.bias != nullptr ? A.bias[n] : 0.f;
    for (int t = t0 + (tid >> 7); t < t1 && m0 + t < A.M; t += 2) {
      const uint32_t at = sW + (t * 128 + row) * 4;
      float sum = 0.f;
      for (int r = 0; r < A.split; ++r) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(map_rank(at, r)) : "memory");
        sum += x;
      }
      sum += bias;
      if (VEDA_IN_BOUNDS(m0 + t < A.M && n < A.N)) {
        if constexpr (sizeof(TO) == 4) out[(m0 + t) * A.ldo + n] = sum;
        else out[(m0 + t) * A.ldo + n] = __float2bfloat16_rn(sum);
      }
    }
  }
  cluster_sync();   // nobody leaves while its partial sums are read
}

namespace {

template <int BN, typename TO>
cudaError_t gemm_run(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, GemmArgs a, int sms,
                     cudaStream_t s) {
  using C = GemmCfg<BN>;
  auto kernel = gemm_fp8_kernel<BN, TO>;
  static SmemLimit limit;
  static std::atomic<int> regs{0};
  cudaError_t e = limit.allow(kernel, C::kSmem);
  if (e != cudaSuccess) return e;
  // The register split (128 threads at 56, 256 at 224) must fit what the block
  // is launched with, or the raise would wait forever.
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
    regs.store(attr.numRegs, std::memory_order_relaxed);
  }
  if (128 * 56 + 256 * 224 > C::kThreads * regs.load(std::memory_order_relaxed)) return cudaErrorInvalidConfiguration;
  a.tiles_m = (a.M + 255) / 256;
  a.tiles_n = (a.N + BN - 1) / BN;
  a.tiles = a.tiles_m * a.tiles_n;
  kernel<<<2u * (unsigned)std::min(a.tiles, sms / 2), C::kThreads, C::kSmem, s>>>(ta, tb, tc, a);
  return cudaGetLastError();
}

template <int TN, typename TO>
cudaError_t gemm_few_run(const CUtensorMap& tx, const CUtensorMap& tw, GemmArgs a, cudaStream_t s) {
  using C = FewCfg<TN>;
  auto kernel = gemm_few_kernel<TN, TO>;
  static SmemLimit limit;
  const cudaError_t e = limit.allow(kernel, C::kSmem);
  if (e != cudaSuccess) return e;
  a.tiles_n = a.nblocks;
  a.tiles_m = (a.M + TN - 1) / TN;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)a.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.tiles_n * a.tiles_m * a.split));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, tx, tw, a);
}

template <typename TO>
cudaError_t gemm_launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const GemmArgs& a, int sms,
                        cudaStream_t s) {
  switch (a.few) {
    case 16: return gemm_few_run<16, TO>(ta, tb, a, s);
    case 32: return gemm_few_run<32, TO>(ta, tb, a, s);
    case 64: return gemm_few_run<64, TO>(ta, tb, a, s);
    default: return a.bn == 128 ? gemm_run<128, TO>(ta, tb, tc, a, sms, s) : gemm_run<256, TO>(ta, tb, tc, a, sms, s);
  }
}

}  // namespace

// Columns of a tile: 128 where such tiles fit the pairs of SMs in one go, since
// a block's chain is shorter then (us, 256 / 128 columns: 14.3 / 12.2 for 777 x
// 2,056 x 1,552, 27.0 / 23.3 for 256 x 5,120 x 5,120); otherwise 256, since an
// SM takes in half as much again per multiplication with 128 (12.9 / 16.7 for
// 1,560 x 1,536 x 1,536, 142 / 218 for 5,000 x 5,120 x 5,120).
inline int gemm_bn(int M, int N, int sms) {
  return ((M + 255LL) / 256) * ((N + 127LL) / 128) * 2 <= sms ? 128 : 256;
}

// Chooses the kernel -- few = 0: tiles of 256 x bn; otherwise the rows per tile of
// the one for few rows -- and into how many CTAs a tile's k blocks are split.
// Measured on 148 SMs with weights that are not in L2, us, few rows at the better
// split / tiles (256 x 128 where these fit in one go):
//   N, K =   15,360, 5,120   5,120, 5,120   4,608, 1,536   1,536, 1,536
//   M =   1:   18.7 / 36.8    10.7 / 25.8     6.7 / 11.7     4.9 / 11.0
//   M =  64:   23.8 / 32.2    14.3 / 23.7    10.1 / 11.7     7.1 / 11.4
//   M = 128:   33.9 / 32.6    20.6 / 24.1    11.3 / 12.1     8.4 / 11.9    64-row tiles: 240, 80, 72, 24
//   M = 192:   59.4 / 33.3    21.4 / 24.0    13.2 / 12.1     9.8 / 11.9                  360, 120, 108, 36
//   M = 256:   62.3 / 33.6    31.3 / 24.3    13.5 / 12.2     9.9 / 11.8                  480, 160, 144, 48
//   M = 512:    116 / 58.8    52.5 / 29.4    16.9 / 12.5    11.9 / 11.9                  960, 320, 288, 96
// So up to 64 rows, and with more while 64-row tiles fill at most 5/9 of the
// SMs (82 of them); above that the better one depends on K, by 12% at most (120
// and 108 tiles above).  Splits are worth it up to 5/3 CTAs per SM.
void plan_gemm_fp8(GemmArgs* a, int sms) {
  a->few = 0;
  a->split = 1;
  a->bn = gemm_bn(a->M, a->N, sms);
  const long long tiles64 = a->nblocks * ((a->M + 63LL) / 64);
  if (a->M > 64 && tiles64 * 9 > sms * 5LL) return;
  a->few = a->M <= 16 ? 16 : a->M <= 32 ? 32 : 64;
  while (a->split < 8 && tiles64 * a->split * 6 <= sms * 5LL && a->kblocks >= 2 * a->split) a->split *= 2;
}

cudaError_t launch_gemm_fp8(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const GemmArgs& a,
                            int out_type, int sms, cudaStream_t s) {
  return out_type == VEDA_FP32 ? gemm_launch<float>(ta, tb, tc, a, sms, s)
                               : gemm_launch<__nv_bfloat16>(ta, tb, tc, a, sms, s);
}

}  // namespace veda
