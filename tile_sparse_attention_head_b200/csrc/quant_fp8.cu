// Operands of the 8-bit product: activations in e4m3 with a scale per row and
// 128 channels, weights in e4m3 with a scale per 128 x 128 block (the rule is
// in layer_common.cuh).
//
// Activations are read through (batch, token, head) strides, so the attention's
// output goes from grid order [B, heads, N, d] to the product's row order
// [B*N, heads*d] in the pass that quantises it.  HBM is the bound: half a warp
// holds one block of 128 channels of a row in registers, takes its maximum
// with four shuffles and writes 128 bytes.  A CTA covers 64 rows of one block of
// channels -- in grid order one contiguous run of a head -- and neighbouring
// CTAs the other blocks of the same rows, so whole output rows are written
// close together.  32,760 x 1,536 bf16 takes 28 to 32 us (5.4 to 4.7 TB/s), 77% of
// the issue slots: the quotient, the maximum across lanes and the conversions.
// A weight of 15,360 x 5,120, laid out once, takes 76 to 86 us.
#include "layer_common.cuh"
#include "kernels.h"
#undef VEDA_SRC_ID
#define VEDA_SRC_ID 10   // bounds-check site id of this file (debug builds)

namespace veda {

constexpr int kQuantRows = 64;   // rows per CTA, four per half-warp

template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const __grid_constant__ QuantArgs A) {
  const int blocks = (A.C + 127) / 128;
  const int kb = blockIdx.x % blocks;
  const int r0 = blockIdx.x / blocks * kQuantRows + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  const int c = kb * 128 + l * 8;
  const bool in_c = c < A.C;
  const T* x = static_cast<const T*>(A.x) + (in_c ? (c / A.d) * A.sh + c % A.d : 0);
  Words<T> w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = r0 + 16 * i;
    if (in_c && row < A.rows) {
      const int b = A.by_n.div(row), n = row - b * (int)A.N;
      const uint4* p = reinterpret_cast<const uint4*>(x + b * A.sb + n * A.sn);
#pragma unroll
      for (int k = 0; k < (int)(sizeof(T) / 2); ++k) w[i].u[k] = __ldcs(p + k);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = r0 + 16 * i;
    const bool here = in_c && row < A.rows;
    uint64_t v[4];
    to_pairs(w[i], v);
    float a = kTiny;
    if (here) a = max_abs(a, v);
#pragma unroll
    for (int off = 8; off; off >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
    if (here && VEDA_IN_BOUNDS(row < A.rows && c + 8 <= A.C)) {
      *reinterpret_cast<uint2*>(A.q + (long long)row * A.C + c) = to_e4m3(v, e4m3_factor(a));
      if (l == 0 && VEDA_IN_BOUNDS(kb < blocks)) A.scale[kb * A.rows + row] = e4m3_scale(a);
    }
  }
}

// One CTA per 128 x 128 block of w [N, K].
template <typename T>
__global__ void __launch_bounds__(256) quant_weight_kernel(const T* __restrict__ w, int N, int K, uint8_t* q,
                                                           float* scale) {
  __shared__ float red[8];
  const int kbs = (K + 127) / 128, nb = blockIdx.x / kbs, kb = blockIdx.x % kbs;
  const int c = kb * 128 + (threadIdx.x & 15) * 8, n0 = nb * 128 + (threadIdx.x >> 4);
  uint64_t v[8][4];
  float a = kTiny;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 16 * i;
    if (n < N && c < K) {
      load_pairs(w + (long long)n * K + c, v[i]);
      a = max_abs(a, v[i]);
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 8; ++k) a = max_nan(a, red[k]);
  const float f = e4m3_factor(a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 16 * i;
    if (n < N && c < K && VEDA_IN_BOUNDS(n < N && c + 8 <= K))
      *reinterpret_cast<uint2*>(q + (long long)n * K + c) = to_e4m3(v[i], f);
  }
  if (threadIdx.x == 0 && VEDA_IN_BOUNDS(nb < (N + 127) / 128 && kb < kbs)) scale[blockIdx.x] = e4m3_scale(a);
}

cudaError_t launch_quant_rows(QuantArgs a, int type, cudaStream_t s) {
  a.by_n = FastDiv((uint32_t)a.N);
  const long long grid = (a.rows + kQuantRows - 1) / kQuantRows * ((a.C + 127) / 128);
  if (type == VEDA_BF16) quant_rows_kernel<__nv_bfloat16><<<(unsigned)grid, 256, 0, s>>>(a);
  else if (type == VEDA_FP16) quant_rows_kernel<__half><<<(unsigned)grid, 256, 0, s>>>(a);
  else quant_rows_kernel<float><<<(unsigned)grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_quant_weight(const void* w, int type, int N, int K, uint8_t* q, float* scale, cudaStream_t s) {
  const unsigned grid = (unsigned)(((N + 127) / 128) * ((K + 127) / 128));
  if (type == VEDA_BF16) quant_weight_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(w), N, K, q, scale);
  else if (type == VEDA_FP16) quant_weight_kernel<<<grid, 256, 0, s>>>(static_cast<const __half*>(w), N, K, q, scale);
  else quant_weight_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(w), N, K, q, scale);
  return cudaGetLastError();
}

}  // namespace veda
