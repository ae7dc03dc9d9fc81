// Residual addition with RMS norm, forward (output in the sublayer's type or
// in e4m3 with a scale per row and 128 channels) and backward.
//
//   h = TX(x + delta)                    stored in the residual stream's type
//   rstd = (mean_c h^2 + eps)^(-1/2),    y = h rstd w
//   g = dy w,  c = mean_c(g h) rstd^2,   dx = d_delta = dh + rstd (g - h c),
//   dw = sum_rows dy h rstd
//
// The norm is taken of the stored h, not of the unrounded sum: backward reads
// h back and then works with exactly the numbers forward normalised, so the
// weight's gradient in fp32 is not limited by a 16-bit rounding between them.
// rstd is computed again from h: its sum shares the other's barrier, and nothing
// has to be kept.  Sums and the statistics are fp32; h, y, dx and d_delta are rounded once.
//
// Every operand is read once and written once, so HBM is the bound.  A row is
// held in registers between the sum and the output, by a group of as many warps
// as it needs (one for up to 512 channels); groups stay and step over the rows.
// The rows to come are on their way to shared memory meanwhile, so loads stay
// in flight through the reduction's barrier and the stores.
//
// Measured (6,548 GB/s is the rate of a plain copy): 75,600 x 5,120 bf16 with
// e4m3 output 440 to 500 us between GPUs (6.2 to 5.4 TB/s); 32,760 x 1,536, fp32
// stream beside bf16: forward 94 us (5.9 TB/s), backward 119 to 127 us (6.4 to 6.0
// TB/s).  Before the arithmetic ran on pairs the 8-bit form was bound by issue
// slots (37 instructions a channel, now 22, half of them a row's fixed part).
//
// dw: each group sums its own rows in registers, a CTA adds its groups in shared
// memory and writes one partial row, and a second kernel adds the partial rows,
// all in a fixed order.  No atomics, so a rerun gives the same bits.
#include "layer_common.cuh"
#include "kernels.h"
#undef VEDA_SRC_ID
#define VEDA_SRC_ID 8   // bounds-check site id of this file (debug builds)

namespace veda {

// Rows in flight per group: what fits two CTAs of 16-bit rows on an SM.
__host__ __device__ constexpr int norm_depth(int cpt) { return cpt == 4 ? 1 : 3; }
__host__ __device__ constexpr int norm_bwd_depth(int cpt) { return cpt == 4 ? 1 : 2; }

template <typename TX, typename TD, int CPT, bool FP8>
__global__ void __launch_bounds__(512) add_rms_norm_kernel(const __grid_constant__ NormArgs A) {
  constexpr int D = norm_depth(CPT);
  __shared__ float red[kRowRed];
  extern __shared__ uint4 ring_raw[];
  const RowGroup g(A.warps);
  const Ring<TX, CPT> rx(ring_raw);
  const Ring<TD, CPT> rd(ring_raw + D * Ring<TX, CPT>::kBytes / 16 * blockDim.x);
  const int nchunk = A.C / 8, slot_size = CPT * blockDim.x;
  const RowPieces<TX, CPT> px(g.t, g.tpt, nchunk);
  const RowPieces<TD, CPT> pd(g.t, g.tpt, nchunk);
  const bool has_delta = A.delta != nullptr, has_h = A.h != nullptr;
  uint64_t w[CPT][4];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = g.t + i * g.tpt;
    if (c < nchunk) load_pairs(A.w + 8 * c, w[i]);
  }
  const float inv_c = 1.f / (float)A.C;
  const long long step = (long long)gridDim.x * g.groups;
  long long row = (long long)blockIdx.x * g.groups + g.group;
  const TX* x = static_cast<const TX*>(A.x) + row * A.ldx;              // D rows ahead
  const TD* delta = static_cast<const TD*>(A.delta) + row * A.ldd;
  TX* h = static_cast<TX*>(A.h) + row * A.C + 8 * g.t;
  using TY = typename std::conditional<FP8, uint8_t, TD>::type;
  TY* y = static_cast<TY*>(A.y) + row * A.C + 8 * g.t;
  float* scale = A.scale + (g.t >> 4) * A.rows;
  auto fetch = [&](long long r, int slot) {
    if (r < A.rows) {
      px.fetch(rx, slot, x);
      if (has_delta) pd.fetch(rd, slot, delta);
    }
    cp_async_commit();
    x += step * A.ldx;
    delta += step * A.ldd;
  };
#pragma unroll 1
  for (int s = 0; s < D; ++s) fetch(row + s * step, s * slot_size);
  for (int turn = 0, slot = 0; row < A.rows; row += step, turn ^= 1) {
    Words<TX> hw[CPT];
    cp_async_wait<D - 1>();
    rx.sync();
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      hw[i] = rx.read(slot, i);
      if (has_delta) add_to(hw[i], rd.read(slot, i));
    }
    rx.sync();
    fetch(row + D * step, slot);
    slot = slot + slot_size == D * slot_size ? 0 : slot + slot_size;
    uint64_t v[CPT][4];
    uint64_t ss = 0;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      to_pairs(hw[i], v[i]);
      if (g.t + i * g.tpt < nchunk) {
        if (has_h && VEDA_IN_BOUNDS(row < A.rows && 8 * (g.t + i * g.tpt) + 8 <= A.C))
          store_words(h + 8 * i * g.tpt, hw[i], A.wide);
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = f2_fma(v[i][k], v[i][k], ss);
      }
    }
    const float rstd = rsqrtf(row_sum(g, f2_sum(ss), red, turn) * inv_c + A.eps);
    const uint64_t rr = f2_all(rstd);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const bool in = g.t + i * g.tpt < nchunk;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] = f2_mul(f2_mul(v[i][k], rr), w[i][k]);
      if constexpr (FP8) {
        // Chunks c .. c+15 of an aligned half-warp are one block of 128 channels.
        float a = kTiny;
        if (in) a = max_abs(a, v[i]);
#pragma unroll
        for (int off = 8; off; off >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
        if (in && VEDA_IN_BOUNDS(row < A.rows && 8 * (g.t + i * g.tpt) + 8 <= A.C)) {
          *reinterpret_cast<uint2*>(y + 8 * i * g.tpt) = to_e4m3(v[i], e4m3_factor(a));
          if ((g.lane & 15) == 0 && VEDA_IN_BOUNDS((g.t >> 4) + 2 * g.W * i < (A.C + 127) / 128))
            scale[2 * g.W * i * A.rows + row] = e4m3_scale(a);
        }
      } else {
        if (in && VEDA_IN_BOUNDS(row < A.rows && 8 * (g.t + i * g.tpt) + 8 <= A.C))
          store_pairs(y + 8 * i * g.tpt, v[i], A.wide);
      }
    }
    h += step * A.C;
    y += step * A.C;
  }
}

template <typename TX, typename TD, int CPT>
__global__ void __launch_bounds__(512) add_rms_norm_bwd_kernel(const __grid_constant__ NormBwdArgs A) {
  constexpr int D = norm_bwd_depth(CPT);
  __shared__ float red[kRowRed];
  extern __shared__ uint4 ring_raw[];
  const RowGroup g(A.warps);
  const Ring<TX, CPT> rh(ring_raw), rdh(ring_raw + D * Ring<TX, CPT>::kBytes / 16 * blockDim.x);
  const Ring<TD, CPT> rdy(ring_raw + 2 * D * Ring<TX, CPT>::kBytes / 16 * blockDim.x);
  const int nchunk = A.C / 8, slot_size = CPT * blockDim.x;
  const RowPieces<TX, CPT> px(g.t, g.tpt, nchunk);
  const RowPieces<TD, CPT> pd(g.t, g.tpt, nchunk);
  const bool has_dh = A.dh != nullptr, has_dx = A.dx != nullptr, has_dd = A.ddelta != nullptr;
  uint64_t w[CPT][4], acc[CPT][4];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = g.t + i * g.tpt;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[i][k] = 0;
    if (c < nchunk) load_pairs(A.w + 8 * c, w[i]);
  }
  const float inv_c = 1.f / (float)A.C;
  const long long step = (long long)gridDim.x * g.groups;
  long long row = (long long)blockIdx.x * g.groups + g.group;
  long long ahead = row * A.C, here = ahead + 8 * g.t;   // elements: D rows ahead, this row's chunk 0
  auto fetch = [&](long long r, int slot) {
    if (r < A.rows) {
      px.fetch(rh, slot, static_cast<const TX*>(A.h) + ahead);
      pd.fetch(rdy, slot, static_cast<const TD*>(A.dy) + ahead);
      if (has_dh) px.fetch(rdh, slot, static_cast<const TX*>(A.dh) + ahead);
    }
    cp_async_commit();
    ahead += step * A.C;
  };
#pragma unroll 1
  for (int s = 0; s < D; ++s) fetch(row + s * step, s * slot_size);
  for (int turn = 0, slot = 0; row < A.rows; row += step, turn ^= 1) {
    uint64_t hv[CPT][4], gv[CPT][4];
    Words<TX> dv[CPT];
    cp_async_wait<D - 1>();
    rh.sync();
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      to_pairs(rh.read(slot, i), hv[i]);
      to_pairs(rdy.read(slot, i), gv[i]);
      if (has_dh) dv[i] = rdh.read(slot, i);
    }
    rh.sync();
    fetch(row + D * step, slot);
    slot = slot + slot_size == D * slot_size ? 0 : slot + slot_size;
    uint64_t hh = 0, gh = 0;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      if (g.t + i * g.tpt < nchunk) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hh = f2_fma(hv[i][k], hv[i][k], hh);
          gh = f2_fma(f2_mul(gv[i][k], w[i][k]), hv[i][k], gh);
        }
      }
    }
    float s1 = f2_sum(hh), s2 = f2_sum(gh);
    row_sum2(g, s1, s2, red, turn);
    const float rstd = rsqrtf(s1 * inv_c + A.eps);
    const uint64_t rr = f2_all(rstd), cc = f2_all(-s2 * inv_c * rstd * rstd);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      if (g.t + i * g.tpt < nchunk) {
        uint64_t d[4] = {0, 0, 0, 0};
        if (has_dh) to_pairs(dv[i], d);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc[i][k] = f2_fma(f2_mul(gv[i][k], rr), hv[i][k], acc[i][k]);
          d[k] = f2_fma(rr, f2_fma(hv[i][k], cc, f2_mul(gv[i][k], w[i][k])), d[k]);
        }
        if (VEDA_IN_BOUNDS(row < A.rows && here == row * A.C + 8 * g.t && 8 * (g.t + i * g.tpt) + 8 <= A.C)) {
          if (has_dx) store_pairs(static_cast<TX*>(A.dx) + here + 8 * i * g.tpt, d, A.wide);
          if (has_dd) store_pairs(static_cast<TD*>(A.ddelta) + here + 8 * i * g.tpt, d, A.wide);
        }
      }
    }
    here += step * A.C;
  }
  if (A.part == nullptr) return;
  cp_async_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring_raw);   // [groups, C], over the ring
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = g.t + i * g.tpt;
    if (c < nchunk) store_shared(sums + g.group * A.C + 8 * c, acc[i]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < A.C; c += blockDim.x) {
    float s = 0.f;
    for (int k = 0; k < g.groups; ++k) s += sums[k * A.C + c];
    if (VEDA_IN_BOUNDS((int)blockIdx.x < A.parts)) A.part[(long long)blockIdx.x * A.C + c] = s;
  }
}

// out[c] = sum_p part[p, c] in a fixed order: warp w of a CTA adds rows w,
// w + 32, ... of its 32 columns, then the 32 sums are added in order.
// blockIdx.y: one of several such sums.
__global__ void __launch_bounds__(1024) sum_partials_kernel(const __grid_constant__ SumArgs A) {
  __shared__ float s[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  const float* part = A.part[blockIdx.y];
  float a = 0.f;
  if (c < A.C) {
#pragma unroll 4
    for (int p = warp; p < A.parts; p += 32) a += part[(long long)p * A.C + c];
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < A.C) {
    float r = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) r += s[k][lane];
    A.out[blockIdx.y][c] = r;
  }
}

cudaError_t launch_sum_partials(const SumArgs& a, int n, cudaStream_t s) {
  sum_partials_kernel<<<dim3((a.C + 31) / 32, n), 1024, 0, s>>>(a);
  return cudaGetLastError();
}

namespace {

RowSplit norm_split(int C, long long rows, int sms) {
  return row_split(C / 8, rows, sms, C <= 256 ? 1 : C <= 8192 ? 2 : 4);
}
long long norm_ctas(long long rows, const RowSplit& r) { return (rows + r.groups - 1) / r.groups; }

template <typename TX, typename TD, int CPT, bool FP8>
cudaError_t norm_fwd(const NormArgs& a, const RowSplit& r, int sms, cudaStream_t s) {
  const auto kernel = add_rms_norm_kernel<TX, TD, CPT, FP8>;
  const size_t smem = (size_t)norm_depth(CPT) * (Ring<TX, CPT>::kBytes + Ring<TD, CPT>::kBytes) * r.threads;
  static SmemLimit limit;
  const cudaError_t e = limit.allow(kernel, smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = resident_ctas(norm_ctas(a.rows, r), kernel, r.threads, smem, sms);
  kernel<<<grid, r.threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename TX, typename TD>
cudaError_t norm_fwd(const NormArgs& a, bool fp8, const RowSplit& r, int sms, cudaStream_t s) {
  if (r.cpt == 1) return fp8 ? norm_fwd<TX, TD, 1, true>(a, r, sms, s) : norm_fwd<TX, TD, 1, false>(a, r, sms, s);
  if (r.cpt == 2) return fp8 ? norm_fwd<TX, TD, 2, true>(a, r, sms, s) : norm_fwd<TX, TD, 2, false>(a, r, sms, s);
  return fp8 ? norm_fwd<TX, TD, 4, true>(a, r, sms, s) : norm_fwd<TX, TD, 4, false>(a, r, sms, s);
}

template <typename TX, typename TD, int CPT>
cudaError_t norm_bwd(NormBwdArgs a, const RowSplit& r, int sms, cudaStream_t s) {
  const auto kernel = add_rms_norm_bwd_kernel<TX, TD, CPT>;
  const size_t smem = (size_t)norm_bwd_depth(CPT) * (2 * Ring<TX, CPT>::kBytes + Ring<TD, CPT>::kBytes) * r.threads;
  static SmemLimit limit;
  cudaError_t e = limit.allow(kernel, smem);
  if (e != cudaSuccess) return e;
  const long long want = std::min(norm_ctas(a.rows, r), (long long)kBwdCtasPerSm * sms);
  const unsigned grid = resident_ctas(want, kernel, r.threads, smem, sms);
  a.parts = (int)grid;
  kernel<<<grid, r.threads, smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.part == nullptr) return e;
  SumArgs sum;
  sum.part[0] = a.part;
  sum.out[0] = a.dw;
  sum.parts = a.parts;
  sum.C = a.C;
  return launch_sum_partials(sum, 1, s);
}

template <typename TX, typename TD>
cudaError_t norm_bwd(const NormBwdArgs& a, const RowSplit& r, int sms, cudaStream_t s) {
  if (r.cpt == 1) return norm_bwd<TX, TD, 1>(a, r, sms, s);
  if (r.cpt == 2) return norm_bwd<TX, TD, 2>(a, r, sms, s);
  return norm_bwd<TX, TD, 4>(a, r, sms, s);
}

}  // namespace

cudaError_t launch_add_rms_norm(NormArgs a, int tx, int td, bool fp8, int sms, cudaStream_t s) {
  const RowSplit r = norm_split(a.C, a.rows, sms);
  a.warps = r.W;
  a.wide = (tx != VEDA_FP32 || on_32_bytes(a.h)) && (td != VEDA_FP32 || fp8 || on_32_bytes(a.y));
  if (tx == VEDA_BF16) return norm_fwd<__nv_bfloat16, __nv_bfloat16>(a, fp8, r, sms, s);
  if (tx == VEDA_FP16) return norm_fwd<__half, __half>(a, fp8, r, sms, s);
  if (td == VEDA_FP32) return norm_fwd<float, float>(a, fp8, r, sms, s);
  return norm_fwd<float, __nv_bfloat16>(a, fp8, r, sms, s);
}

// Partial rows of dw at most: one per CTA.
int add_rms_norm_bwd_parts(long long rows, int C, int sms) {
  return (int)std::min(norm_ctas(rows, norm_split(C, rows, sms)), (long long)kBwdCtasPerSm * sms);
}

cudaError_t launch_add_rms_norm_bwd(NormBwdArgs a, int tx, int td, int sms, cudaStream_t s) {
  const RowSplit r = norm_split(a.C, a.rows, sms);
  a.warps = r.W;
  a.wide = (tx != VEDA_FP32 || on_32_bytes(a.dx)) && (td != VEDA_FP32 || on_32_bytes(a.ddelta));
  if (tx == VEDA_BF16) return norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, r, sms, s);
  if (tx == VEDA_FP16) return norm_bwd<__half, __half>(a, r, sms, s);
  if (td == VEDA_FP32) return norm_bwd<float, float>(a, r, sms, s);
  return norm_bwd<float, __nv_bfloat16>(a, r, sms, s);
}

}  // namespace veda
