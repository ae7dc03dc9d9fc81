// Matrix product in 8-bit floating point with a scale for each block of 128:
//
//   C[m, n] = sum_kb sa[kb, m] sb[n / 128, kb] sum_{k in block kb} A[m, k] B[n, k]  (+ bias[n])
//
// A [M, K] and B [N, K] are e4m3, sa one fp32 scale per row and 128 channels,
// sb one per 128 x 128 block; C is bf16 or fp32.  The inner sums run on the
// tensor cores (tcgen05, kind::f8f6f4, fp32 accumulation); each block's sum
// leaves tensor memory once and is scaled and added into fp32 registers.
//
// One persistent CTA per SM walks 128 x BN tiles.  A producer warp brings one
// 128-byte-wide k block of A and B per step into a ring of shared-memory stages
// by TMA (K tails and edge rows are filled with zeros, which add nothing); an
// issuer warp multiplies the stage into one of two tensor-memory buffers; two
// warpgroups, each with half the columns, add buffer after buffer into their
// registers while the next block is multiplied.
#include "layer_common.cuh"
#include "kernels.h"
#undef VEDA_SRC_ID
#define VEDA_SRC_ID 11   // bounds-check site id of this file (debug builds)

namespace veda {

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 operands, fp32 accumulate, K = 32.
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: e4m3 A/B (format 0), fp32 D, both K-major.
__host__ __device__ constexpr uint32_t make_idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int BN>
struct GemmCfg {
  static constexpr int kThreads = 384;
  static constexpr int kStages = 4;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = BN * 128;
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffBar = kOffB + kStages * kBBytes;
  static constexpr int kOffMisc = kOffBar + 16 * 8;
  static constexpr size_t kSmem = 1024 + kOffMisc + 64;
  static constexpr uint32_t kTmemCols = 2 * BN;
};

enum {
  GBAR_FULL = 0,    // +stage (4)
  GBAR_EMPTY = 4,   // +stage (4)
  GBAR_DFULL = 8,   // +buffer (2)
  GBAR_DFREE = 10,  // +buffer (2)
  GBAR_DRAIN = 12
};

__device__ __forceinline__ bool gemm_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, timeout_ns));
}

// Tile t in an order that keeps a wave's operands in L2: groups of 16 tile
// rows, column by column inside a group.
__device__ __forceinline__ void gemm_tile(const GemmArgs& A, int t, int* m, int* n) {
  const int per_group = 16 * A.tiles_n;
  const int first = t / per_group * 16, r = t % per_group;
  const int rows = min(16, A.tiles_m - first);
  *m = first + r % rows;
  *n = r / rows;
}

template <int BN, typename TO>
__global__ void __launch_bounds__(384, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ GemmArgs A) {
  using C = GemmCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sA = smem_u32(smem), sB = smem_u32(smem + C::kOffB), bar0 = smem_u32(smem + C::kOffBar);
  auto bar = [&](int b) { return bar0 + 8u * (uint32_t)b; };
  int* misc = reinterpret_cast<int*>(smem + C::kOffMisc);   // [0] tmem base, [1] abort
  volatile int* abort = misc + 1;
  const uint64_t tmo = A.timeout_ns;

  if (tid == 0) {
    misc[1] = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(GBAR_FULL + s), 1);
      mbar_init(bar(GBAR_EMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(GBAR_DFULL + s), 1);
      mbar_init(bar(GBAR_DFREE + s), 8);
    }
    mbar_init(bar(GBAR_DRAIN), 1);
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

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      int it = 0;
      bool ok = true;
      if (lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
      }
      for (int t = blockIdx.x; ok && t < A.tiles; t += gridDim.x) {
        int m, n;
        gemm_tile(A, t, &m, &n);
        for (int kb = 0; kb < A.kblocks; ++kb) {
          const int st = it % C::kStages, fill = it / C::kStages;
          if (fill >= 1 && !(ok = gemm_wait(bar(GBAR_EMPTY + st), (fill - 1) & 1, abort, tmo))) break;
          if (lane == 0 && VEDA_IN_BOUNDS(m * 128 < A.M && n * BN < A.N && kb * 128 < A.K)) {
            mbar_arrive_expect_tx(bar(GBAR_FULL + st), C::kABytes + C::kBBytes);
            tma_load_2d(sA + st * C::kABytes, &tmA, bar(GBAR_FULL + st), kb * 128, m * 128);
            tma_load_2d(sB + st * C::kBBytes, &tmB, bar(GBAR_FULL + st), kb * 128, n * BN);
          }
          __syncwarp();
          ++it;
        }
      }
      if (*abort) {
        int dummy = 0;
        for (int i = it > C::kStages ? it - C::kStages : 0; i < it; ++i)
          mbar_wait(bar(GBAR_FULL + i % C::kStages), (i / C::kStages) & 1, &dummy, tmo);
      }
    } else if (warp == 1) {
      constexpr uint32_t idesc = make_idesc_e4m3(128, BN);
      const uint64_t da0 = make_sdesc_sw128(sA, 16, 1024), db0 = make_sdesc_sw128(sB, 16, 1024);
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < A.tiles; t += gridDim.x) {
        for (int kb = 0; kb < A.kblocks; ++kb, ++it) {
          const int st = it % C::kStages, buf = it & 1;
          if (!(ok = gemm_wait(bar(GBAR_FULL + st), (it / C::kStages) & 1, abort, tmo))) break;
          if (it >= 2 && !(ok = gemm_wait(bar(GBAR_DFREE + buf), ((it >> 1) - 1) & 1, abort, tmo))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t da = da0 + (uint64_t)((st * C::kABytes) >> 4), db = db0 + (uint64_t)((st * C::kBBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f8_ss(tmem + buf * BN, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
            umma_commit(bar(GBAR_EMPTY + st));
            umma_commit(bar(GBAR_DFULL + buf));
          }
          __syncwarp();
        }
      }
      if (lane == 0) umma_commit(bar(GBAR_DRAIN));
      __syncwarp();
      int dummy = 0;
      mbar_wait(bar(GBAR_DRAIN), 0, &dummy, tmo);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    constexpr int HN = BN / 2;               // columns of this warpgroup
    const int half = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * HN);
    int it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < A.tiles; t += gridDim.x) {
      int m, n;
      gemm_tile(A, t, &m, &n);
      const int row = m * 128 + quarter * 32 + lane, col0 = n * BN + half * HN;
      const bool has_row = row < A.M;
      const float* sa = A.sa + (has_row ? row : 0);
      const float* sb = A.sb + (long long)min(col0 / 128, A.nblocks - 1) * A.kblocks;
      uint64_t acc[HN / 2];
#pragma unroll
      for (int j = 0; j < HN / 2; ++j) acc[j] = 0;
      float scale = sa[0] * sb[0];
      for (int kb = 0; kb < A.kblocks; ++kb, ++it) {
        const int buf = it & 1;
        const float next = kb + 1 < A.kblocks ? sa[(long long)(kb + 1) * A.M] * sb[kb + 1] : 0.f;
        if (!(ok = gemm_wait(bar(GBAR_DFULL + buf), (it >> 1) & 1, abort, tmo))) break;
        tc_fence_after();
        const uint64_t s2 = f2(scale, scale);
#pragma unroll
        for (int c = 0; c < HN; c += 64) {
          float v[64];
          tmem_ld32(t_lane + buf * BN + c, v);
          tmem_ld32(t_lane + buf * BN + c + 32, v + 32);
          tmem_ld_wait();
          if (c + 64 >= HN) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(GBAR_DFREE + buf));
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c / 2 + j] = f2_fma(f2(v[2 * j], v[2 * j + 1]), s2, acc[c / 2 + j]);
        }
        scale = next;
      }
      if (ok && has_row) {
        TO* out = static_cast<TO*>(A.out) + (long long)row * A.ldo;
#pragma unroll
        for (int j = 0; j < HN / 8; ++j) {
          const int col = col0 + 8 * j;
          if (col >= A.N) break;
          if (A.bias != nullptr) {
            uint64_t b[4];
            load_pairs(A.bias + col, b);
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[4 * j + k] = f2_add(acc[4 * j + k], b[k]);
          }
          if (VEDA_IN_BOUNDS(row < A.M && col + 8 <= A.N)) store_pairs(out + col, acc + 4 * j);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

namespace {

template <int BN, typename TO>
cudaError_t gemm_run(const CUtensorMap& ta, const CUtensorMap& tb, GemmArgs a, int sms, cudaStream_t s) {
  using C = GemmCfg<BN>;
  auto kernel = gemm_fp8_kernel<BN, TO>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  // The register split (128 threads at 56, 256 at 224) must fit what the block
  // is launched with, or the raise would wait forever.
  cudaFuncAttributes attr;
  if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
  if (128 * 56 + 256 * 224 > C::kThreads * attr.numRegs) return cudaErrorInvalidConfiguration;
  a.tiles_m = (a.M + 127) / 128;
  a.tiles_n = (a.N + BN - 1) / BN;
  a.tiles = a.tiles_m * a.tiles_n;
  kernel<<<(unsigned)std::min(a.tiles, sms), C::kThreads, C::kSmem, s>>>(ta, tb, a);
  return cudaGetLastError();
}

}  // namespace

// Rows of the A and B boxes that the launch below wants for a problem.
void gemm_fp8_boxes(const GemmArgs& a, int* rows_a, int* rows_b) {
  (void)a;
  *rows_a = 128;
  *rows_b = 256;
}

cudaError_t launch_gemm_fp8(const CUtensorMap& ta, const CUtensorMap& tb, const GemmArgs& a, int out_type, int sms,
                            cudaStream_t s) {
  return out_type == VEDA_FP32 ? gemm_run<256, float>(ta, tb, a, sms, s)
                               : gemm_run<256, __nv_bfloat16>(ta, tb, a, sms, s);
}

}  // namespace veda
