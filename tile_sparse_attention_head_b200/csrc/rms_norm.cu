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
// Sums and the statistics are fp32; h, y, dx and d_delta are rounded once.
//
// Every operand is read once and written once, so HBM is the bound.  A row is
// held in registers between the sum and the output.  Rows of up to 1,024
// channels take one warp each (four rows per CTA, no barrier), longer ones a
// CTA of as many warps as the row needs; CTAs stay and step over the rows,
// with the weights kept in registers.
//
// dw: each CTA (each warp for short rows) sums its own rows in registers and
// writes one partial row; a second kernel adds the partial rows in a fixed
// order.  No atomics, so a rerun gives the same bits.
#include "layer_common.cuh"
#include "kernels.h"
#undef VEDA_SRC_ID
#define VEDA_SRC_ID 8   // bounds-check site id of this file (debug builds)

namespace veda {

template <typename TX, typename TD, int CPT, bool FP8>
__global__ void __launch_bounds__(512) add_rms_norm_kernel(const __grid_constant__ NormArgs A) {
  __shared__ float red[64];
  const int W = A.warps;                        // warps per row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_cta = W == 1 ? (int)(blockDim.x >> 5) : 1;
  const int t = W == 1 ? lane : threadIdx.x;
  const int tpt = 32 * W, nchunk = A.C / 8;
  const TX* x = static_cast<const TX*>(A.x);
  const TD* delta = static_cast<const TD*>(A.delta);
  TX* h = static_cast<TX*>(A.h);
  float w[CPT][8];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * tpt;
    if (c < nchunk) load8(A.w + 8 * c, w[i]);
  }
  const float inv_c = 1.f / (float)A.C;
  int turn = 0;
  for (long long row = (long long)blockIdx.x * per_cta + (W == 1 ? warp : 0); row < A.rows;
       row += (long long)gridDim.x * per_cta, turn ^= 1) {
    float v[CPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (c < nchunk && VEDA_IN_BOUNDS(row < A.rows)) load8(x + row * A.ldx + 8 * c, v[i]);
    }
    if (delta != nullptr) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int c = t + i * tpt;
        if (c < nchunk) {
          float d[8];
          load8(delta + row * A.ldd + 8 * c, d);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] = round_to<TX>(v[i][k] + d[k]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (c < nchunk) {
        if (h != nullptr) store8(h + row * A.C + 8 * c, v[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(v[i][k], v[i][k], ss);
      }
    }
    ss = W == 1 ? warp_sum(ss) : cta_sum(ss, red, W, warp, lane, turn);
    const float rstd = rsqrtf(ss * inv_c + A.eps);
    if (A.rstd != nullptr && t == 0) A.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      float y[8];
      if (c < nchunk) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = v[i][k] * rstd * w[i][k];
      }
      if constexpr (FP8) {
        // Chunks c .. c+15 of an aligned half-warp are one block of 128 channels.
        uint32_t m = kTinyBits;
        if (c < nchunk) {
#pragma unroll
          for (int k = 0; k < 8; ++k) m = max(m, abs_bits(y[k]));
        }
#pragma unroll
        for (int off = 8; off; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float a = __uint_as_float(m);
        if (c < nchunk) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(A.y) + row * A.C + 8 * c) = pack_e4m3x8(y, kE4M3Max / a);
          if ((c & 15) == 0) A.scale[(long long)(c >> 4) * A.rows + row] = a / kE4M3Max;
        }
      } else {
        if (c < nchunk) store8(static_cast<TD*>(A.y) + row * A.C + 8 * c, y);
      }
    }
  }
}

template <typename TX, typename TD, int CPT>
__global__ void __launch_bounds__(512) add_rms_norm_bwd_kernel(const __grid_constant__ NormBwdArgs A) {
  __shared__ float red[64];
  const int W = A.warps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_cta = W == 1 ? (int)(blockDim.x >> 5) : 1;
  const int t = W == 1 ? lane : threadIdx.x;
  const int tpt = 32 * W, nchunk = A.C / 8;
  const TX* h = static_cast<const TX*>(A.h);
  const TX* dh = static_cast<const TX*>(A.dh);
  const TD* dy = static_cast<const TD*>(A.dy);
  float w[CPT][8], acc[CPT][8];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * tpt;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;
    if (c < nchunk) load8(A.w + 8 * c, w[i]);
  }
  const float inv_c = 1.f / (float)A.C;
  int turn = 0;
  const long long first = (long long)blockIdx.x * per_cta + (W == 1 ? warp : 0);
  for (long long row = first; row < A.rows; row += (long long)gridDim.x * per_cta, turn ^= 1) {
    float hv[CPT][8], g[CPT][8];
    float s = 0.f;
    const float rstd = A.rstd[row];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (c < nchunk && VEDA_IN_BOUNDS(row < A.rows)) {
        load8(h + row * A.C + 8 * c, hv[i]);
        load8(dy + row * A.C + 8 * c, g[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (c < nchunk) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          acc[i][k] = fmaf(g[i][k] * rstd, hv[i][k], acc[i][k]);
          g[i][k] *= w[i][k];
          s = fmaf(g[i][k], hv[i][k], s);
        }
      }
    }
    s = W == 1 ? warp_sum(s) : cta_sum(s, red, W, warp, lane, turn);
    const float c1 = s * inv_c * rstd * rstd;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (c < nchunk) {
        float d[8];
        if (dh != nullptr) {
          load8(dh + row * A.C + 8 * c, d);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = fmaf(rstd, g[i][k] - hv[i][k] * c1, d[k]);
        if (A.dx != nullptr) store8(static_cast<TX*>(A.dx) + row * A.C + 8 * c, d);
        if (A.ddelta != nullptr) store8(static_cast<TD*>(A.ddelta) + row * A.C + 8 * c, d);
      }
    }
  }
  if (A.part != nullptr) {
    const long long p = (long long)blockIdx.x * per_cta + (W == 1 ? warp : 0);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (c < nchunk && VEDA_IN_BOUNDS(p < A.parts)) store8(A.part + p * A.C + 8 * c, acc[i]);
    }
  }
}

// out[c] = sum_p part[p, c] in a fixed order: warp w of a CTA adds rows w,
// w + 32, ... of its 32 columns, then the 32 sums are added in order.
__global__ void __launch_bounds__(1024) sum_partials_kernel(const float* __restrict__ part, int parts, int C,
                                                            float* __restrict__ out) {
  __shared__ float s[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < C) {
#pragma unroll 4
    for (int p = warp; p < parts; p += 32) a += part[(long long)p * C + c];
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < C) {
    float r = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) r += s[k][lane];
    out[c] = r;
  }
}

cudaError_t launch_sum_partials(const float* part, int parts, int C, float* out, cudaStream_t s) {
  sum_partials_kernel<<<(C + 31) / 32, 1024, 0, s>>>(part, parts, C, out);
  return cudaGetLastError();
}

namespace {

// Chunks per thread and warps per row for rows of nchunk chunks.
struct RowSplit {
  int cpt, warps, threads, per_cta;
};
RowSplit row_split(int nchunk, int max_cpt) {
  RowSplit r;
  if (nchunk <= 32 * max_cpt) {
    r.cpt = nchunk <= 32 ? 1 : nchunk <= 64 ? 2 : 4;
    r.warps = 1;
  } else {
    r.cpt = nchunk <= 512 * 2 ? 2 : 4;
    r.warps = (nchunk + 32 * r.cpt - 1) / (32 * r.cpt);
  }
  r.threads = r.warps == 1 ? 128 : 32 * r.warps;
  r.per_cta = r.warps == 1 ? 4 : 1;
  return r;
}

template <typename TX, typename TD>
cudaError_t norm_fwd(const NormArgs& a, bool fp8, const RowSplit& r, unsigned grid, cudaStream_t s) {
#define VEDA_NORM(CPT)                                                                    \
  if (r.cpt == CPT) {                                                                     \
    if (fp8) add_rms_norm_kernel<TX, TD, CPT, true><<<grid, r.threads, 0, s>>>(a);        \
    else add_rms_norm_kernel<TX, TD, CPT, false><<<grid, r.threads, 0, s>>>(a);           \
  }
  VEDA_NORM(1) else VEDA_NORM(2) else VEDA_NORM(4)
#undef VEDA_NORM
  return cudaGetLastError();
}

template <typename TX, typename TD>
cudaError_t norm_bwd(const NormBwdArgs& a, const RowSplit& r, unsigned grid, cudaStream_t s) {
  if (r.cpt == 1) add_rms_norm_bwd_kernel<TX, TD, 1><<<grid, r.threads, 0, s>>>(a);
  else if (r.cpt == 2) add_rms_norm_bwd_kernel<TX, TD, 2><<<grid, r.threads, 0, s>>>(a);
  else add_rms_norm_bwd_kernel<TX, TD, 4><<<grid, r.threads, 0, s>>>(a);
  return cudaGetLastError();
}

unsigned norm_grid(long long rows, const RowSplit& r, int sms) {
  const long long want = (rows + r.per_cta - 1) / r.per_cta, most = (long long)sms * (2048 / r.threads);
  return (unsigned)(want < most ? want : most);
}

}  // namespace

cudaError_t launch_add_rms_norm(NormArgs a, int tx, int td, bool fp8, int sms, cudaStream_t s) {
  const RowSplit r = row_split(a.C / 8, 4);
  a.warps = r.warps;
  const unsigned grid = norm_grid(a.rows, r, sms);
  if (tx == VEDA_BF16) return norm_fwd<__nv_bfloat16, __nv_bfloat16>(a, fp8, r, grid, s);
  if (tx == VEDA_FP16) return norm_fwd<__half, __half>(a, fp8, r, grid, s);
  if (td == VEDA_FP32) return norm_fwd<float, float>(a, fp8, r, grid, s);
  return norm_fwd<float, __nv_bfloat16>(a, fp8, r, grid, s);
}

// Partial rows of dw: one per CTA, or per warp where a warp has a row.
int add_rms_norm_bwd_parts(long long rows, int C, int sms) {
  const RowSplit r = row_split(C / 8, 2);
  return (int)norm_grid(rows, r, sms) * r.per_cta;
}

cudaError_t launch_add_rms_norm_bwd(NormBwdArgs a, int tx, int td, float* dw, int sms, cudaStream_t s) {
  const RowSplit r = row_split(a.C / 8, 2);
  a.warps = r.warps;
  a.parts = add_rms_norm_bwd_parts(a.rows, a.C, sms);
  const unsigned grid = norm_grid(a.rows, r, sms);
  cudaError_t e;
  if (tx == VEDA_BF16) e = norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, r, grid, s);
  else if (tx == VEDA_FP16) e = norm_bwd<__half, __half>(a, r, grid, s);
  else if (td == VEDA_FP32) e = norm_bwd<float, float>(a, r, grid, s);
  else e = norm_bwd<float, __nv_bfloat16>(a, r, grid, s);
  if (e != cudaSuccess || dw == nullptr) return e;
  return launch_sum_partials(a.part, a.parts, a.C, dw, s);
}

}  // namespace veda
