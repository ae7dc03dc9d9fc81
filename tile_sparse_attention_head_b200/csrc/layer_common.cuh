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

// Chunks on their way from global memory, D rows ahead of their use, in shared
// memory.  A thread copies (cp.async, 16 bytes at a time) and reads its own
// chunks only, so nothing has to be synchronised between threads: one commit
// per row, and a wait for all but the D - 1 newest rows before reading.  The
// layout is [slot][chunk][16-byte piece][thread]: no bank conflicts.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int CPT>
struct Ring {
  static constexpr int kPieces = sizeof(T) / 2;
  static constexpr int kBytes = CPT * kPieces * 16;   // per thread and slot
  const uint4* base;
  __device__ __forceinline__ explicit Ring(const void* smem) : base(static_cast<const uint4*>(smem) + threadIdx.x) {}
  __device__ __forceinline__ const uint4* at(int slot, int i, int k) const {
    return base + ((slot * CPT + i) * kPieces + k) * blockDim.x;
  }
  __device__ __forceinline__ void fetch(int slot, int i, const T* p) const {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) cp_async16(smem_u32(at(slot, i, k)), reinterpret_cast<const uint4*>(p) + k);
  }
  __device__ __forceinline__ void read(int slot, int i, float* v) const {
    uint4 u[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) u[k] = *at(slot, i, k);
    load8(reinterpret_cast<const T*>(u), v);
  }
};

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

// How rows are spread over threads: a row belongs to `W` warps of a CTA (its
// group), `cpt` chunks per thread, and a CTA has up to as many groups as make
// 16 warps.  Thread t of a group has the chunks t, t + 32 W, ...
struct RowSplit {
  int cpt, W, groups, threads;
};
inline RowSplit row_split(int nchunk, long long rows, int sms) {
  RowSplit r;
  r.cpt = nchunk <= 32 ? 1 : nchunk <= 1024 ? 2 : 4;
  r.W = (nchunk + 32 * r.cpt - 1) / (32 * r.cpt);
  r.groups = 16 / r.W;
  const long long each = (rows + sms - 1) / sms;   // few rows: spread them over the SMs first
  if (each < r.groups) r.groups = each < 1 ? 1 : (int)each;
  r.threads = 32 * r.W * r.groups;
  return r;
}

struct RowGroup {
  int W, groups, group, warp, lane, t, tpt;   // warp: within the group
  __device__ __forceinline__ explicit RowGroup(int warps) {
    W = warps;
    groups = (int)(blockDim.x >> 5) / W;
    const int w = threadIdx.x >> 5;
    group = w / W;
    warp = w - group * W;
    lane = threadIdx.x & 31;
    t = warp * 32 + lane;
    tpt = 32 * W;
  }
};

__device__ __forceinline__ void group_sync(const RowGroup& g) {
  if (g.W == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(g.group + 1), "r"(32 * g.W) : "memory");
}

// Sums over the threads of a group, the same in every thread (the addition
// order is fixed).  `red` holds kRowRed floats per CTA; `turn` alternates
// between calls, so that one barrier per call is enough: a warp can only be one
// call ahead of the slowest reader.
constexpr int kRowRed = 16 * 2 * 2 * 16;
__device__ __forceinline__ void row_sum2(const RowGroup& g, float& a, float& b, float* red, int turn) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (g.W == 1) return;
  float* r = red + (g.group * 2 + turn) * 32;
  if (g.lane == 0) {
    r[g.warp] = a;
    r[16 + g.warp] = b;
  }
  group_sync(g);
  a = warp_sum(g.lane < g.W ? r[g.lane] : 0.f);
  b = warp_sum(g.lane < g.W ? r[16 + g.lane] : 0.f);
}
__device__ __forceinline__ float row_sum(const RowGroup& g, float a, float* red, int turn) {
  a = warp_sum(a);
  if (g.W == 1) return a;
  float* r = red + (g.group * 2 + turn) * 32;
  if (g.lane == 0) r[g.warp] = a;
  group_sync(g);
  return warp_sum(g.lane < g.W ? r[g.lane] : 0.f);
}

template <typename K>
inline cudaError_t allow_smem(K kernel, size_t smem) {
  if (smem <= 40 * 1024) return cudaSuccess;   // what any kernel may have beside its static part
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

// CTAs that are resident at once, so that each can keep stepping over rows.
template <typename K>
inline unsigned resident_ctas(K kernel, int threads, size_t smem, int sms) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
  return (unsigned)(n * sms);
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
