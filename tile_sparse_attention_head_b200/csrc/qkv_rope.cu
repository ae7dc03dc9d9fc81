// From the QKV product to the attention's operands: RMS norm of Q and K,
// rotary positions over the grid's three axes, and the change from token order
// [B, N, heads, d] (any strides) to grid order [B, heads, N, d] bf16, in one
// pass; and the backward of it.
//
//   xn = x rstd w,  rstd = (mean x^2 + eps)^(-1/2)   mean over heads*d (row), over d (head), or no norm
//   (a, b) -> (a cos - b sin, a sin + b cos)          for the two channels of a pair
//
// The channels of a head are split into time, height and width (and a rest
// that is not turned); a pair lies inside one axis, as neighbours
// (interleaved) or as the halves of the axis's channels.  cos and sin come from
// one table per axis, so a token's angles are three short rows that stay in L1.
// Backward, with R the rotation:  g = R^T dout,  dw = sum g x rstd,
//   dx = rstd (g w - x mean(g w x) rstd^2).
// rstd is recomputed from x, which backward reads anyway.  Everything between
// the loads and the one rounding at the store is fp32.
//
// HBM is the bound: each element is read once and written once.  A thread owns
// chunks of 8 channels; chunk c of a token belongs to thread c % tpt with tpt
// a multiple of 32, hence of d/8, so a thread meets the same channels of a
// head in all its chunks and fetches its cos and sin once per token.  Stores to
// grid order are whole head rows (128 or 256 bytes).  Tokens of up to 1,024
// channels take a warp each, longer ones a CTA of as many warps as they need.
#include "layer_common.cuh"
#include "kernels.h"
#undef VEDA_SRC_ID
#define VEDA_SRC_ID 9   // bounds-check site id of this file (debug builds)

namespace veda {

// Where the angle of channel `ch` of a head comes from.
struct Angle {
  int axis;      // 0 time, 1 height, 2 width, -1 not turned
  int at;        // column of the axis's table
  int partner;   // the pair's other channel
  bool second;   // whether ch is the pair's second channel
};

__device__ __forceinline__ Angle angle_of(const RopeArgs& A, int ch) {
  Angle g{-1, 0, ch, false};
  int base = 0;
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    const int u = ch - base, dim = A.dim[a];
    if (u >= 0 && u < dim) {
      g.axis = a;
      if (A.halves) {
        const int half = dim >> 1;
        g.second = u >= half;
        g.at = g.second ? u - half : u;
        g.partner = g.second ? ch - half : ch + half;
      } else {
        g.second = u & 1;
        g.at = u >> 1;
        g.partner = ch ^ 1;
      }
    }
    base += dim;
  }
  return g;
}

// Per-thread addresses of the angles of its 8 channels: HALVES needs one angle
// per channel, neighbours share one.
template <bool HALVES>
struct Turn {
  static constexpr int kN = HALVES ? 8 : 4;
  const float2* base[kN];
  int step[kN];       // table row length, 0 where the channel is not turned
  int axis[kN];
  int src[HALVES ? 8 : 1];     // partner's place in the warp's scratch
  float sgn[HALVES ? 8 : 1];
  __device__ __forceinline__ void init(const RopeArgs& A, int ch0, int lane, int lanes_per_head) {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const Angle g = angle_of(A, ch0 + (HALVES ? j : 2 * j));
      axis[j] = g.axis;
      step[j] = g.axis < 0 ? 0 : A.dim[g.axis] >> 1;
      base[j] = g.axis < 0 ? nullptr : A.tab[g.axis] + g.at;
      if constexpr (HALVES) {
        const int first = lane / lanes_per_head * lanes_per_head;
        src[j] = (first + (g.partner >> 3)) * 9 + (g.partner & 7);
        sgn[j] = g.second ? 1.f : -1.f;
      }
    }
  }
  __device__ __forceinline__ void load(int t, int y, int x, float2* cs) const {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int pos = axis[j] == 0 ? t : axis[j] == 1 ? y : x;
      cs[j] = axis[j] < 0 ? make_float2(1.f, 0.f) : base[j][pos * step[j]];
    }
  }
  // v turned by +angle (dir = 1) or -angle (dir = -1).  `scratch`: this
  // warp's 32 * 9 floats (a lane's 8 values at 9 * lane: no bank conflicts).
  __device__ __forceinline__ void apply(float* v, const float2* cs, float dir, float* scratch, int lane) const {
    if constexpr (HALVES) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) scratch[lane * 9 + j] = v[j];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float r = fmaf(v[j], cs[j].x, sgn[j] * dir * cs[j].y * scratch[src[j]]);
        v[j] = axis[j] < 0 ? v[j] : r;   // an infinity that is not turned stays one
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j], b = v[2 * j + 1], s = dir * cs[j].y;
        v[2 * j] = axis[j] < 0 ? a : fmaf(a, cs[j].x, -b * s);
        v[2 * j + 1] = axis[j] < 0 ? b : fmaf(a, s, b * cs[j].x);
      }
    }
  }
};

__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int off = lanes >> 1; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A.order[blockIdx.y]: 0 = Q, 1 = K, 2 = V (V is only moved).
template <typename T, int CPT, bool HALVES>
__global__ void __launch_bounds__(512) qkv_rope_kernel(const __grid_constant__ RopeArgs A) {
  __shared__ float red[64];
  extern __shared__ float scratch_all[];
  const int which = A.order[blockIdx.y];
  const int W = A.warps, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_cta = W == 1 ? (int)(blockDim.x >> 5) : 1;
  const int t = W == 1 ? lane : threadIdx.x;
  const int tpt = 32 * W, lph = A.d / 8, nchunk = A.heads * lph;
  const int ch0 = (t % lph) * 8, head0 = t / lph, head_step = tpt / lph;
  const int norm = which == 2 ? VEDA_NORM_NONE : A.norm;
  const T* in = static_cast<const T*>(A.in[which]);
  const long long sb = A.sb[which], sn = A.sn[which], sh = A.sh[which];
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(A.out[which]);
  float* scratch = scratch_all + warp * (32 * 9);
  Turn<HALVES> turn;
  turn.init(A, ch0, lane, lph);
  float w[CPT][8];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * tpt;
    if (norm != VEDA_NORM_NONE && c < nchunk) load8(A.w[which] + (norm == VEDA_NORM_ROW ? 8 * c : ch0), w[i]);
  }
  const float inv_n = 1.f / (float)(norm == VEDA_NORM_ROW ? A.heads * A.d : A.d);
  int flip = 0;
  for (long long tok = (long long)blockIdx.x * per_cta + (W == 1 ? warp : 0); tok < A.tokens;
       tok += (long long)gridDim.x * per_cta, flip ^= 1) {
    const int b = (int)(tok / A.N), n = (int)(tok % A.N);
    const T* row = in + b * sb + n * sn;
    float v[CPT][8];
    float r[CPT];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (c < nchunk && VEDA_IN_BOUNDS(tok < A.tokens)) {
        load8(row + (head0 + i * head_step) * sh + ch0, v[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
      }
    }
    float2 cs[Turn<HALVES>::kN];
    if (which < 2) turn.load(n / (A.H * A.W), n / A.W % A.H, n % A.W, cs);
    if (norm != VEDA_NORM_NONE) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(v[i][k], v[i][k], s);
        r[i] = s;
        ss += s;
      }
      if (norm == VEDA_NORM_ROW) {
        ss = W == 1 ? warp_sum(ss) : cta_sum(ss, red, W, warp, lane, flip);
        ss = rsqrtf(ss * inv_n + A.eps);
#pragma unroll
        for (int i = 0; i < CPT; ++i) r[i] = ss;
      } else {
#pragma unroll
        for (int i = 0; i < CPT; ++i) r[i] = rsqrtf(head_sum(r[i], lph) * inv_n + A.eps);
      }
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (norm != VEDA_NORM_NONE && c < nchunk) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] *= r[i] * w[i][k];
      }
      if (which < 2) turn.apply(v[i], cs, 1.f, scratch, lane);
      if (c < nchunk && VEDA_IN_BOUNDS(head0 + i * head_step < A.heads))
        store8(out + (((long long)b * A.heads + head0 + i * head_step) * A.N + n) * A.d + ch0, v[i]);
    }
  }
}

template <typename T, int CPT, bool HALVES>
__global__ void __launch_bounds__(512) qkv_rope_bwd_kernel(const __grid_constant__ RopeArgs A) {
  __shared__ float red[64];
  extern __shared__ float scratch_all[];
  const int which = A.order[blockIdx.y];
  const int W = A.warps, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_cta = W == 1 ? (int)(blockDim.x >> 5) : 1;
  const int t = W == 1 ? lane : threadIdx.x;
  const int tpt = 32 * W, lph = A.d / 8, nchunk = A.heads * lph;
  const int ch0 = (t % lph) * 8, head0 = t / lph, head_step = tpt / lph;
  const int norm = which == 2 ? VEDA_NORM_NONE : A.norm;
  const T* in = static_cast<const T*>(A.in[which]);
  const long long sb = A.sb[which], sn = A.sn[which], sh = A.sh[which];
  const __nv_bfloat16* dout = static_cast<const __nv_bfloat16*>(A.out[which]);
  T* dx = static_cast<T*>(A.dx[which]);
  const long long dsb = A.dsb[which], dsn = A.dsn[which], dsh = A.dsh[which];
  float* scratch = scratch_all + warp * (32 * 9);
  Turn<HALVES> turn;
  turn.init(A, ch0, lane, lph);
  float w[CPT][8], acc[CPT][8];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * tpt;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = w[i][k] = 0.f;
    if (norm != VEDA_NORM_NONE && c < nchunk) load8(A.w[which] + (norm == VEDA_NORM_ROW ? 8 * c : ch0), w[i]);
  }
  const float inv_n = 1.f / (float)(norm == VEDA_NORM_ROW ? A.heads * A.d : A.d);
  for (long long tok = (long long)blockIdx.x * per_cta + (W == 1 ? warp : 0); tok < A.tokens;
       tok += (long long)gridDim.x * per_cta) {
    const int b = (int)(tok / A.N), n = (int)(tok % A.N);
    float g[CPT][8], v[CPT][8];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt, hd = head0 + i * head_step;
#pragma unroll
      for (int k = 0; k < 8; ++k) g[i][k] = v[i][k] = 0.f;
      if (c < nchunk && VEDA_IN_BOUNDS(hd < A.heads)) {
        load8(dout + (((long long)b * A.heads + hd) * A.N + n) * A.d + ch0, g[i]);
        if (norm != VEDA_NORM_NONE) load8(in + b * sb + n * sn + hd * sh + ch0, v[i]);
      }
    }
    if (which < 2) {
      float2 cs[Turn<HALVES>::kN];
      turn.load(n / (A.H * A.W), n / A.W % A.H, n % A.W, cs);
#pragma unroll
      for (int i = 0; i < CPT; ++i) turn.apply(g[i], cs, -1.f, scratch, lane);
    }
    if (norm != VEDA_NORM_NONE) {
      float s1[CPT], s2[CPT];
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        s1[i] = s2[i] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          s1[i] = fmaf(v[i][k], v[i][k], s1[i]);
          s2[i] = fmaf(g[i][k] * w[i][k], v[i][k], s2[i]);
        }
      }
      if (norm == VEDA_NORM_ROW) {
        float a = 0.f, c = 0.f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) a += s1[i], c += s2[i];
        if (W == 1) {
          a = warp_sum(a);
          c = warp_sum(c);
        } else {
          // two sums per token: each has its own half of `red`, and the
          // second's barrier stands between the first's next use and its readers
          a = cta_sum(a, red, W, warp, lane, 0);
          c = cta_sum(c, red, W, warp, lane, 1);
        }
#pragma unroll
        for (int i = 0; i < CPT; ++i) s1[i] = a, s2[i] = c;
      } else {
#pragma unroll
        for (int i = 0; i < CPT; ++i) s1[i] = head_sum(s1[i], lph), s2[i] = head_sum(s2[i], lph);
      }
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const float rstd = rsqrtf(s1[i] * inv_n + A.eps), c1 = s2[i] * inv_n * rstd * rstd;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          acc[i][k] = fmaf(g[i][k] * rstd, v[i][k], acc[i][k]);
          g[i][k] = rstd * (g[i][k] * w[i][k] - v[i][k] * c1);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (c < nchunk) store8(dx + b * dsb + n * dsn + (head0 + i * head_step) * dsh + ch0, g[i]);
    }
  }
  float* part = A.part[which];
  if (norm == VEDA_NORM_NONE || part == nullptr) return;   // CTA-uniform
  if (norm == VEDA_NORM_ROW) {
    const long long p = (long long)blockIdx.x * per_cta + (W == 1 ? warp : 0);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * tpt;
      if (c < nchunk && VEDA_IN_BOUNDS(p < A.parts)) store8(part + p * (A.heads * A.d) + 8 * c, acc[i]);
    }
  } else {
    // One weight row for all heads: add the thread's chunks, the lanes that
    // share channels, then the warps in order.
    float a[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] = 0.f;
#pragma unroll
      for (int i = 0; i < CPT; ++i) a[k] += acc[i][k];
      for (int off = 16; off >= lph; off >>= 1) a[k] += __shfl_xor_sync(0xffffffffu, a[k], off);
    }
    float* all = scratch_all;   // d floats per warp (at most 128 of the warp's 288)
    __syncthreads();
    if (lane < lph) {
#pragma unroll
      for (int k = 0; k < 8; ++k) all[warp * 288 + lane * 8 + k] = a[k];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < A.d; c += blockDim.x) {
      float s = 0.f;
      for (int k = 0; k < (int)(blockDim.x >> 5); ++k) s += all[k * 288 + c];
      if (VEDA_IN_BOUNDS((int)blockIdx.x < A.parts)) part[(long long)blockIdx.x * A.d + c] = s;
    }
  }
}

// (cos, sin) of (start + step i) theta^(-2j/dim), angles in fp64: at position
// 10^4 an fp32 angle is already off by half a thousandth.
__global__ void rope_table_kernel(int n, int pairs, int dim, double log2_theta, double start, double step, float2* out) {
  const long long e = blockIdx.x * (long long)blockDim.x + threadIdx.x;
  if (e >= (long long)n * pairs) return;
  const int i = (int)(e / pairs), j = (int)(e % pairs);
  const double a = (start + step * i) * exp2(-2.0 * j / dim * log2_theta);
  double s, c;
  sincos(a, &s, &c);
  out[e] = make_float2((float)c, (float)s);
}

namespace {

struct TokenSplit {
  int cpt, warps, threads, per_cta;
  size_t smem;
};
TokenSplit token_split(int nchunk, int max_cpt) {
  TokenSplit r;
  if (nchunk <= 32 * max_cpt) {
    r.cpt = nchunk <= 32 ? 1 : nchunk <= 64 ? 2 : 4;
    r.warps = 1;
  } else {
    r.cpt = nchunk <= 512 * 2 ? 2 : 4;
    r.warps = (nchunk + 32 * r.cpt - 1) / (32 * r.cpt);
  }
  r.threads = r.warps == 1 ? 128 : 32 * r.warps;
  r.per_cta = r.warps == 1 ? 4 : 1;
  r.smem = (size_t)(r.threads / 32) * 32 * 9 * sizeof(float);
  return r;
}

unsigned rope_grid(long long tokens, const TokenSplit& r, int sms) {
  const long long want = (tokens + r.per_cta - 1) / r.per_cta, most = (long long)sms * (2048 / r.threads);
  return (unsigned)(want < most ? want : most);
}

template <typename T, bool HALVES>
cudaError_t rope_run(const RopeArgs& a, const TokenSplit& r, dim3 grid, bool backward, cudaStream_t s) {
  const size_t smem = HALVES || backward ? r.smem : 0;
#define VEDA_ROPE(CPT)                                                                          \
  if (r.cpt == CPT) {                                                                           \
    if (backward) qkv_rope_bwd_kernel<T, CPT, HALVES><<<grid, r.threads, smem, s>>>(a);         \
    else qkv_rope_kernel<T, CPT, HALVES><<<grid, r.threads, smem, s>>>(a);                      \
  }
  VEDA_ROPE(1) else VEDA_ROPE(2) else VEDA_ROPE(4)
#undef VEDA_ROPE
  return cudaGetLastError();
}

template <typename T>
cudaError_t rope_pairing(const RopeArgs& a, const TokenSplit& r, dim3 grid, bool backward, cudaStream_t s) {
  return a.halves ? rope_run<T, true>(a, r, grid, backward, s) : rope_run<T, false>(a, r, grid, backward, s);
}

cudaError_t rope_types(const RopeArgs& a, int type, const TokenSplit& r, dim3 grid, bool backward, cudaStream_t s) {
  if (type == VEDA_BF16) return rope_pairing<__nv_bfloat16>(a, r, grid, backward, s);
  if (type == VEDA_FP16) return rope_pairing<__half>(a, r, grid, backward, s);
  return rope_pairing<float>(a, r, grid, backward, s);
}

}  // namespace

cudaError_t launch_qkv_rope(RopeArgs a, int type, int n_which, int sms, cudaStream_t s) {
  const TokenSplit r = token_split(a.heads * a.d / 8, 4);
  a.warps = r.warps;
  return rope_types(a, type, r, dim3(rope_grid(a.tokens, r, sms), n_which), false, s);
}

// Rows of weight-gradient partials, each heads*d (row norm) or d (head norm) floats.
int qkv_rope_bwd_parts(long long tokens, int heads, int d, bool row, int sms) {
  const TokenSplit r = token_split(heads * d / 8, 2);
  return (int)rope_grid(tokens, r, sms) * (row ? r.per_cta : 1);
}

cudaError_t launch_qkv_rope_bwd(RopeArgs a, int type, int n_which, float* const* dw, int sms, cudaStream_t s) {
  const TokenSplit r = token_split(a.heads * a.d / 8, 2);
  a.warps = r.warps;
  a.parts = qkv_rope_bwd_parts(a.tokens, a.heads, a.d, a.norm == VEDA_NORM_ROW, sms);
  cudaError_t e = rope_types(a, type, r, dim3(rope_grid(a.tokens, r, sms), n_which), true, s);
  if (e != cudaSuccess || a.norm == VEDA_NORM_NONE) return e;
  const int C = a.norm == VEDA_NORM_ROW ? a.heads * a.d : a.d;
  for (int i = 0; i < n_which; ++i) {
    const int which = a.order[i];
    if (which == 2 || dw[which] == nullptr) continue;
    if ((e = launch_sum_partials(a.part[which], a.parts, C, dw[which], s)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_rope_table(int n, int dim, double theta, double start, double step, float* out, cudaStream_t s) {
  const long long e = (long long)n * (dim / 2);
  rope_table_kernel<<<(unsigned)((e + 255) / 256), 256, 0, s>>>(n, dim / 2, dim, log2(theta), start, step,
                                                                reinterpret_cast<float2*>(out));
  return cudaGetLastError();
}

}  // namespace veda
