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

#include <atomic>
#include <mutex>
#include <type_traits>

#include "veda_common.cuh"

namespace veda {

// A chunk as it lies in memory, and as four pairs of fp32 (the arithmetic runs
// on pairs: one issue slot for two channels).
template <typename T>
struct Words {
  uint4 u[sizeof(T) / 2];
};
__device__ __forceinline__ void to_pairs(const Words<float>& x, uint64_t* p) {
  p[0] = f2(__uint_as_float(x.u[0].x), __uint_as_float(x.u[0].y));
  p[1] = f2(__uint_as_float(x.u[0].z), __uint_as_float(x.u[0].w));
  p[2] = f2(__uint_as_float(x.u[1].x), __uint_as_float(x.u[1].y));
  p[3] = f2(__uint_as_float(x.u[1].z), __uint_as_float(x.u[1].w));
}
__device__ __forceinline__ uint64_t bf16_pair(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint64_t fp16_pair(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return f2(f.x, f.y);
}
__device__ __forceinline__ void to_pairs(const Words<__nv_bfloat16>& x, uint64_t* p) {
  p[0] = bf16_pair(x.u[0].x), p[1] = bf16_pair(x.u[0].y), p[2] = bf16_pair(x.u[0].z), p[3] = bf16_pair(x.u[0].w);
}
__device__ __forceinline__ void to_pairs(const Words<__half>& x, uint64_t* p) {
  p[0] = fp16_pair(x.u[0].x), p[1] = fp16_pair(x.u[0].y), p[2] = fp16_pair(x.u[0].z), p[3] = fp16_pair(x.u[0].w);
}

// Pairs rounded to T, nearest even.
template <typename T>
__device__ __forceinline__ Words<T> to_words(const uint64_t* p) {
  Words<T> r;
  if constexpr (sizeof(T) == 4) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) f2_split(p[k], v[2 * k], v[2 * k + 1]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      r.u[k] = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                          __float_as_uint(v[4 * k + 3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a, b;
      f2_split(p[k], a, b);
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[k] = pack_bf16x2(a, b);
      }
    }
    r.u[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void load_pairs(const T* p, uint64_t* v) {
  Words<T> w;
#pragma unroll
  for (int k = 0; k < (int)(sizeof(T) / 2); ++k) w.u[k] = reinterpret_cast<const uint4*>(p)[k];
  to_pairs(w, v);
}
// `wide`: every fp32 output of the launch starts on a 32-byte border (tensors
// need 16).  Then an fp32 chunk is one store, where two of 16 bytes would each
// touch half of every sector.
template <typename T>
__device__ __forceinline__ void store_words(T* p, const Words<T>& w, bool wide) {
  if constexpr (sizeof(T) == 4) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %9, 0;\n\t"
        "@p st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t"
        "@!p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t"
        "@!p st.global.v4.b32 [%0 + 16], {%5, %6, %7, %8};\n\t}" ::"l"(p), "r"(w.u[0].x), "r"(w.u[0].y),
        "r"(w.u[0].z), "r"(w.u[0].w), "r"(w.u[1].x), "r"(w.u[1].y), "r"(w.u[1].z), "r"(w.u[1].w), "r"((int)wide)
        : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = w.u[0];
  }
}
template <typename T>
__device__ __forceinline__ void store_pairs(T* p, const uint64_t* v, bool wide) { store_words(p, to_words<T>(v), wide); }
inline bool on_32_bytes(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

__device__ __forceinline__ void store_shared(float* p, const uint64_t* v) {
  const Words<float> w = to_words<float>(v);
  reinterpret_cast<uint4*>(p)[0] = w.u[0];
  reinterpret_cast<uint4*>(p)[1] = w.u[1];
}

// x + d rounded to x's type.  Of two 16-bit values the sum is exact in fp32, or
// so far from a rounding border that one rounding and two agree, so the 16-bit
// addition (two channels an instruction) gives what an fp32 sum rounded to 16
// bits gives.
template <typename T>
__device__ __forceinline__ uint32_t add_words(uint32_t a, uint32_t b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 r =
        __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
template <typename TX, typename TD>
__device__ __forceinline__ void add_to(Words<TX>& x, const Words<TD>& d) {
  if constexpr (sizeof(TX) == 2) {
    x.u[0] = make_uint4(add_words<TX>(x.u[0].x, d.u[0].x), add_words<TX>(x.u[0].y, d.u[0].y),
                        add_words<TX>(x.u[0].z, d.u[0].z), add_words<TX>(x.u[0].w, d.u[0].w));
  } else {
    uint64_t a[4], b[4];
    to_pairs(x, a);
    to_pairs(d, b);
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = f2_add(a[k], b[k]);
    x = to_words<TX>(a);
  }
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_all(float a) { return f2(a, a); }
__device__ __forceinline__ float f2_sum(uint64_t a) {
  float lo, hi;
  f2_split(a, lo, hi);
  return lo + hi;
}

// Chunks on their way from global memory, D rows ahead of their use, in shared
// memory.  A warp copies (cp.async, 16 bytes at a time) and reads its own
// chunks only, so no barrier is needed: one commit per row, and a wait for all
// but the D - 1 newest rows before reading.  A 16-bit chunk is one piece, which
// its thread copies itself.  An fp32 chunk is two; there lane l copies the
// pieces l and 32 + l of the warp's 64, so that a copy's sectors are whole, and
// the warp synchronises around it.  Piece q lies at q ^ (q / 8 & 1), which
// leaves no bank conflicts.
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

//
// A slot is named by its first chunk's place, slot * CPT * blockDim.x.
template <typename T, int CPT>
struct Ring {
  static constexpr int kPieces = sizeof(T) / 2;
  static constexpr int kBytes = CPT * kPieces * 16;   // per thread and slot
  const uint4* mine;                                  // the warp's part of slot 0, chunk 0
  uint32_t write[kPieces];
  int threads;
  __device__ __forceinline__ explicit Ring(const void* smem) : threads(blockDim.x) {
    const int lane = threadIdx.x & 31;
    mine = static_cast<const uint4*>(smem) + (threadIdx.x - lane) * kPieces;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) write[j] = smem_u32(mine + place(lane + 32 * j));
  }
  __device__ __forceinline__ static int place(int q) { return kPieces == 1 ? q : q ^ (q >> 3 & 1); }
  // The chunk, relative to the thread's own, that its piece j belongs to, and the piece's first channel there.
  __device__ __forceinline__ static int other(int j) {
    const int lane = threadIdx.x & 31;
    return kPieces == 1 ? 0 : ((lane + 32 * j) >> 1) - lane;
  }
  __device__ __forceinline__ static int channel(int j) { return kPieces == 1 ? 0 : (threadIdx.x & 1) * 4; }
  __device__ __forceinline__ void fetch(int slot, int i, int j, const T* p) const {
    cp_async16(write[j] + (slot + i * threads) * (kPieces * 16), p);
  }
  __device__ __forceinline__ Words<T> read(int slot, int i) const {
    Words<T> w;
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
      w.u[j] = mine[(slot + i * threads) * kPieces + place(kPieces * (threadIdx.x & 31) + j)];
    return w;
  }
  // Around the reads of a row: its pieces have come, and may be overwritten.
  __device__ __forceinline__ static void sync() {
    if constexpr (kPieces == 2) __syncwarp();
  }
};

// The pieces that a thread copies of a dense row, as offsets (in elements) from the row's start.
template <typename T, int CPT>
struct RowPieces {
  static constexpr int kPieces = sizeof(T) / 2;
  int off[kPieces], step, valid;
  __device__ __forceinline__ RowPieces(int t, int tpt, int nchunk) : step(8 * tpt), valid(0) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int c = t + Ring<T, CPT>::other(j);
      off[j] = 8 * c + Ring<T, CPT>::channel(j);
#pragma unroll
      for (int i = 0; i < CPT; ++i) valid |= (c + i * tpt < nchunk ? 1 : 0) << (i * kPieces + j);
    }
  }
  __device__ __forceinline__ void fetch(const Ring<T, CPT>& ring, int slot, const T* row) const {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (valid >> (i * kPieces + j) & 1) ring.fetch(slot, i, j, row + (off[j] + i * step));
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// How rows are spread over threads: a row belongs to `W` warps of a CTA (its
// group), `cpt` chunks per thread, and a CTA has up to as many groups as make
// 16 warps (or what the kernel with two chunks per thread has registers for).  Thread t of a group has the chunks t, t + 32 W, ...
struct RowSplit {
  int cpt, W, groups, threads;
};
inline RowSplit row_split(int nchunk, long long rows, int sms, int cpt, int most_warps = 16) {
  RowSplit r;
  r.cpt = cpt;
  r.W = (nchunk + 32 * r.cpt - 1) / (32 * r.cpt);
  r.groups = most_warps / r.W;
  const long long each = (rows + sms - 1) / sms;   // few rows: spread them over the SMs first
  if (each < r.groups) r.groups = each < 1 ? 1 : (int)each;
  r.threads = 32 * r.W * r.groups;
  return r;
}
// Chunks per thread, of 1 to `most`: those that leave the fewest idle, the most
// of them if several do (a row costs a thread some 190 instructions whatever its
// chunks, each chunk 76, in the rotary kernel).
inline int best_cpt(int nchunk, int most) {
  if (nchunk <= 32) return 1;
  int best = 0, best_slots = 0;
  for (int cpt = 2; cpt <= most; ++cpt) {
    const int W = (nchunk + 32 * cpt - 1) / (32 * cpt), slots = W * 32 * cpt;
    if (W <= 16 && (best == 0 || slots <= best_slots)) {
      best = cpt;
      best_slots = slots;
    }
  }
  return best == 0 ? 4 : best;
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

constexpr size_t kMostSmem = 220 * 1024;   // of a CTA, beside a few KB of static shared memory

// A kernel's limit of dynamic shared memory, raised when a launch in that
// device's context first asks for more, and never lowered, so that threads which
// launch with different sizes do not take each other's limit away.  It is not
// raised at once to what any launch may ever need: the driver sizes L1 by it,
// and the norm of 75,600 x 5,120 took 498 us instead of 446 with a limit of 220
// KB.
struct SmemLimit {
  std::mutex mu;
  unsigned long long context[64] = {};
  int most[64] = {};
  template <typename K>
  cudaError_t allow(K kernel, size_t smem) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    const unsigned long long id = current_context_id();
    if (id != 0 && id == context[dev] && most[dev] >= (int)smem) return cudaSuccess;
    const int want = id != 0 && id == context[dev] ? std::max(most[dev], (int)smem) : (int)smem;
    const cudaError_t set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, want);
    if (set == cudaSuccess) {
      context[dev] = current_context_id();   // the call may have made the context
      most[dev] = want;
    }
    return set;
  }
};

// CTAs to launch for `want` of them: at most as many as are resident at once, so
// that each can keep stepping over rows.
template <typename K>
inline unsigned resident_ctas(long long want, K kernel, int threads, size_t smem, int sms) {
  if (want <= sms) return (unsigned)want;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
  return (unsigned)(want < (long long)n * sms ? want : (long long)n * sms);
}

// The 8-bit rule, the norm's and the quantisers' alike: with a a block's largest
// magnitude, but at least 2^-100 (so that a block of zeros has a scale and the
// factor stays finite), its scale is a * (1 / 448) and it holds e4m3(x * f),
// nearest even, with f = 448 / a correctly rounded.  The maximum passes NaN on: a
// block with an infinity or NaN gets a scale that is infinite or NaN, and
// stands for NaN as a whole, rather than for a finite wrong value.
constexpr float kE4M3Max = 448.f;
constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100

__device__ __forceinline__ float e4m3_scale(float a) { return a * (1.f / 448.f); }
__device__ __forceinline__ float e4m3_factor(float a) { return kE4M3Max / a; }

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// The larger of m and the pairs' magnitudes.
__device__ __forceinline__ float max_abs(float m, const uint64_t* p) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a, b;
    f2_split(p[k], a, b);
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
  }
  return m;
}

__device__ __forceinline__ uint2 to_e4m3(const uint64_t* p, float r) {
  const uint64_t rr = f2_all(r);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 v;
    f2_split(f2_mul(p[k], rr), v.x, v.y);
    w[k] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

}  // namespace veda
