// Pieces shared by the operators around the attention (residual and RMS norm,
// 8-bit quantisation, rotary positions): 8-channel vector access in the
// library's element types, block sums, and the e4m3 rule.
//
// All of these kernels are bound by HBM.  A thread owns 8 consecutive channels
// ("a chunk": 16 bytes of a 16-bit type, 32 of fp32) at a time, so every warp
// access covers whole 32-byte sectors whatever the row length.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "veda_common.cuh"

namespace veda {

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __bfloat1622float2(b[k]);
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const __half2* b = reinterpret_cast<const __half2*>(&u);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __half22float2(b[k]);
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float* v) {
  uint4 u;
  __half2* b = reinterpret_cast<__half2*>(&u);
#pragma unroll
  for (int k = 0; k < 4; ++k) b[k] = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
  *reinterpret_cast<uint4*>(p) = u;
}

// v rounded to T and back: the value a stored element stands for.
template <typename T>
__device__ __forceinline__ float round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ float round_to<__nv_bfloat16>(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }
template <>
__device__ __forceinline__ float round_to<__half>(float v) { return __half2float(__float2half_rn(v)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sum over the `warps` warps of the CTA, the same value in every thread (the
// addition order is fixed).  `red` holds 2 x 32 floats; `turn` alternates
// between calls, so one barrier per call is enough: a warp can only be one
// call ahead of the slowest reader.
__device__ __forceinline__ float cta_sum(float v, float* red, int warps, int warp, int lane, int turn) {
  v = warp_sum(v);
  if (lane == 0) red[turn * 32 + warp] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[turn * 32 + lane] : 0.f);
}

// The 8-bit rule: a block's scale is s = a / 448 with a its largest magnitude,
// but at least 2^-100 (so that a block of zeros has a scale and 448 / a stays
// finite), and the block holds e4m3(x * (448 / a)), nearest even.  The maximum
// runs on the magnitudes' bit patterns, which order like the magnitudes and
// put infinity and then NaN on top: a block with either gets a scale that is
// infinite or NaN, and stands for NaN as a whole, rather than passing on a
// finite wrong value.
constexpr float kE4M3Max = 448.f;
constexpr uint32_t kTinyBits = (127u - 100u) << 23;   // 2^-100

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint2 pack_e4m3x8(const float* v, float r) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * k] * r, v[2 * k + 1] * r), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

}  // namespace veda
