// Matrix product in 8-bit floating point with a scale for each block of 128:
//
//   C[m, n] = sum_kb sa[kb, m] sb[n / 128, kb] sum_{k in block kb} A[m, k] B[n, k]  (+ bias[n])
//
// A [M, K] and B [N, K] are e4m3, sa one fp32 scale per row and 128 channels,
// sb one per 128 x 128 block; C is bf16 or fp32.  The inner sums run on the
// tensor cores (tcgen05, kind::f8f6f4, fp32 accumulation); each block's sum
// leaves tensor memory once and is scaled and added into fp32 registers.
//
// Two CTAs on neighbouring SMs (a cluster) work on one 256 x 256 tile: each
// brings its 128 rows of A and half of B's rows, and one instruction multiplies
// on both (cta_group::2).  So an SM takes in 32 KB per k block instead of the
// 48 KB that a 128 x 256 tile of its own would need -- at 512 cycles of tensor
// work per block, 64 bytes a cycle, which is what an SM can take from L2.
//
// Pairs stay and walk the tiles.  A producer warp per CTA brings one
// 128-byte-wide k block of A and B per step into a ring of shared-memory stages
// by TMA (K tails and edge rows are filled with zeros, which add nothing); an
// issuer warp in the pair's first CTA multiplies the stage into one of two
// tensor-memory buffers; in both CTAs two warpgroups, each with half the
// columns, add buffer after buffer into their registers while the next block is
// multiplied.  The scales come ahead by cp.async.  Results leave through shared
// memory and TMA stores, which drop what lies past M and N.
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
// No release at cluster scope: it would wait for the thread's copies in flight.
// What has to be ordered are tensor-memory reads, by tcgen05.fence before it.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
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

// Shared memory of the main kernel.
struct GemmCfg {
  static constexpr int kThreads = 384;
  static constexpr int kStages = 4;
  static constexpr int kAhead = 8;                    // scales in flight per thread
  static constexpr int kHalf = 128 * 128;             // a CTA's part of A, or of B, per stage
  static constexpr int kOffB = kStages * kHalf;
  static constexpr int kOffOut = 2 * kStages * kHalf; // per consumer warp two pieces of 32 rows x 128 bytes
  static constexpr int kOffScale = kOffOut + 8 * 2 * 4096;
  static constexpr int kOffBar = kOffScale + kAhead * 256 * 8;
  static constexpr int kOffMisc = kOffBar + 16 * 8;
  static constexpr size_t kSmem = 1024 + kOffMisc + 64;
};

enum {
  GBAR_FULL = 0,    // +stage (4): both CTAs' operands have come (the first CTA's barrier counts)
  GBAR_EMPTY = 4,   // +stage (4)
  GBAR_DFULL = 8,   // +buffer (2)
  GBAR_DFREE = 10,  // +buffer (2): both CTAs' consumers have read it (the first CTA's barrier counts)
};

__device__ __forceinline__ bool gemm_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, timeout_ns));
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

template <typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(384, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmC, const __grid_constant__ GemmArgs A) {
  using C = GemmCfg;
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
      mbar_init(bar(GBAR_EMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(GBAR_DFULL + s), 1);
      mbar_init(bar(GBAR_DFREE + s), 16);
    }
    fence_mbar_init();
  }
  if (warp == 1) pair::tmem_alloc(smem_u32(&misc[0]), 512);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      int it = 0;
      bool ok = true;
      if (lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmC);
      }
      for (int t = first_tile; ok && t < A.tiles; t += pairs) {
        int m, n;
        gemm_tile(A, t, &m, &n);
        const int row = m * 256 + rank * 128, col = n * 256 + rank * 128;
        for (int kb = 0; kb < A.kblocks; ++kb) {
          const int st = it % C::kStages, fill = it / C::kStages;
          if (fill >= 1 && !(ok = gemm_wait(bar(GBAR_EMPTY + st), (fill - 1) & 1, abort, tmo))) break;
          if (lane == 0 && VEDA_IN_BOUNDS(m * 256 < A.M && n * 256 < A.N && kb * 128 < A.K)) {
            const uint32_t full = map_rank(bar(GBAR_FULL + st), 0);
            if (rank == 0) mbar_arrive_expect_tx(bar(GBAR_FULL + st), 4 * C::kHalf);
            pair::tma_load_2d(sA + st * C::kHalf, &tmA, full, kb * 128, row);
            pair::tma_load_2d(sB + st * C::kHalf, &tmB, full, kb * 128, col);
          }
          __syncwarp();
          ++it;
        }
      }
      // The last fills: on a failure the copies in flight are waited for (at
      // the barriers that count them); otherwise the signals that they were
      // used, the last things to come to this CTA's barriers from outside.
      int dummy = 0;
      const bool failed = *abort != 0;
      for (int i = it > C::kStages ? it - C::kStages : 0; i < it && !(failed && rank); ++i)
        mbar_wait(bar((failed ? GBAR_FULL : GBAR_EMPTY) + i % C::kStages), (i / C::kStages) & 1, &dummy, tmo);
    } else if (warp == 1 && rank == 0) {
      constexpr uint32_t idesc = make_idesc_e4m3(256, 256);
      const uint64_t da0 = make_sdesc_sw128(sA, 16, 1024), db0 = make_sdesc_sw128(sB, 16, 1024);
      int it = 0;
      bool ok = true;
      for (int t = first_tile; ok && t < A.tiles; t += pairs) {
        for (int kb = 0; kb < A.kblocks; ++kb, ++it) {
          const int st = it % C::kStages, buf = it & 1;
          if (!(ok = gemm_wait(bar(GBAR_FULL + st), (it / C::kStages) & 1, abort, tmo))) break;
          if (it >= 2 && !(ok = gemm_wait(bar(GBAR_DFREE + buf), ((it >> 1) - 1) & 1, abort, tmo))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t step = (uint64_t)((st * C::kHalf) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              pair::umma_f8(tmem + buf * 256, da0 + step + 2 * kk, db0 + step + 2 * kk, idesc, kk > 0 ? 1u : 0u);
            pair::umma_commit(bar(GBAR_EMPTY + st));
            pair::umma_commit(bar(GBAR_DFULL + buf));
          }
          __syncwarp();
        }
      }
      // The consumers have seen the last commit, or a wait ran out; then the
      // multiplications in flight are waited for here, again with a limit.
      if (!ok && it > 0) {
        int dummy = 0;
        mbar_wait(bar(GBAR_DFULL + ((it - 1) & 1)), ((it - 1) >> 1) & 1, &dummy, tmo);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    constexpr int HN = 128;                  // columns of this warpgroup
    constexpr int PC = 128 / sizeof(TO);     // columns of an output piece
    const int half = (warp - 4) >> 2, quarter = warp & 3, ctid = tid - 128;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * HN);
    const uint32_t free0 = map_rank(bar(GBAR_DFREE), 0);
    float* scales = reinterpret_cast<float*>(smem + C::kOffScale) + 2 * ctid;   // [kAhead][256][2]: sa, sb
    uint8_t* out = smem + C::kOffOut + (warp - 4) * 8192;
    // Where the scales ahead are: tile, block, and the row's and column block's first scale.
    int at = first_tile, akb = 0, aslot = 0;
    const float *pa = nullptr, *pb = nullptr;
    auto enter = [&]() {
      int m, n;
      gemm_tile(A, at, &m, &n);
      pa = A.sa + min(m * 256 + rank * 128 + quarter * 32 + lane, A.M - 1);
      pb = A.sb + (long long)min(n * 2 + half, A.nblocks - 1) * A.kblocks;
    };
    auto ahead = [&]() {
      if (at < A.tiles) {
        if (akb == 0) enter();
        const uint32_t dst = smem_u32(scales + aslot * 512);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(pa) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + 4), "l"(pb) : "memory");
        pa += A.M;
        ++pb;
        if (++akb == A.kblocks) {
          akb = 0;
          at += pairs;
        }
      }
      cp_async_commit();
      aslot = (aslot + 1) & (C::kAhead - 1);
    };
#pragma unroll 1
    for (int i = 0; i < C::kAhead - 1; ++i) ahead();
    int it = 0, pieces = 0;
    bool ok = true;
    for (int t = first_tile; ok && t < A.tiles; t += pairs) {
      int m, n;
      gemm_tile(A, t, &m, &n);
      uint64_t acc[HN / 2];
#pragma unroll
      for (int j = 0; j < HN / 2; ++j) acc[j] = 0;
      for (int kb = 0; kb < A.kblocks; ++kb, ++it) {
        const int buf = it & 1;
        ahead();
        cp_async_wait<C::kAhead - 1>();
        const float2 sc = *reinterpret_cast<const float2*>(scales + (it & (C::kAhead - 1)) * 512);
        const uint64_t s2 = f2_all(sc.x * sc.y);
        if (!(ok = gemm_wait(bar(GBAR_DFULL + buf), (it >> 1) & 1, abort, tmo))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < HN; c += 64) {
          float v[64];
          tmem_ld32(t_lane + buf * 256 + c, v);
          tmem_ld32(t_lane + buf * 256 + c + 32, v + 32);
          tmem_ld_wait();
          if (c + 64 >= HN) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(free0 + 8u * (uint32_t)buf);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c / 2 + j] = f2_fma(f2(v[2 * j], v[2 * j + 1]), s2, acc[c / 2 + j]);
        }
      }
      const int row0 = m * 256 + rank * 128 + quarter * 32, col0 = n * 256 + half * HN;
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
    cp_async_wait<0>();
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

namespace {

template <typename TO>
cudaError_t gemm_run(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, GemmArgs a, int sms,
                     cudaStream_t s) {
  using C = GemmCfg;
  auto kernel = gemm_fp8_kernel<TO>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  // The register split (128 threads at 56, 256 at 224) must fit what the block
  // is launched with, or the raise would wait forever.
  cudaFuncAttributes attr;
  if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
  if (128 * 56 + 256 * 224 > C::kThreads * attr.numRegs) return cudaErrorInvalidConfiguration;
  a.tiles_m = (a.M + 255) / 256;
  a.tiles_n = (a.N + 255) / 256;
  a.tiles = a.tiles_m * a.tiles_n;
  kernel<<<2u * (unsigned)std::min(a.tiles, sms / 2), C::kThreads, C::kSmem, s>>>(ta, tb, tc, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_fp8(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const GemmArgs& a,
                            int out_type, int sms, cudaStream_t s) {
  return out_type == VEDA_FP32 ? gemm_run<float>(ta, tb, tc, a, sms, s) : gemm_run<__nv_bfloat16>(ta, tb, tc, a, sms, s);
}

}  // namespace veda
