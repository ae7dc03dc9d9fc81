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
// HBM is the bound: each element is read once and written once.  A token's row
// of one operand belongs to a group of warps (as in the norm), which steps over
// the tokens with the next rows on their way to shared memory, first all of Q,
// then K, then V, so that the operand's weights and angle addresses stay in
// registers.  Chunk c of a row belongs to thread c % tpt with tpt a multiple of
// 32, hence of d/8, so a thread meets the same channels of a head in all its
// chunks and reads its cos and sin once per token.  A token's d/2 angles come
// to shared memory with its row, one copy for the group.  Stores to grid order
// are whole head rows (128 or 256 bytes).
//
// Measured (6,548 GB/s is the rate of a plain copy): 75,600 tokens of 40 x 128
// 930 us, 5.0 TB/s; 32,760 tokens of 12 x 128 forward 127 us (4.8 TB/s), backward
// 215 to 221 us (3.5 TB/s).  With halves, whose eight angle places spill above one
// chunk a thread, 1,690, 210 and 325 us.  fp16 input takes what bf16 does, fp32 160
// us forward and 264 us backward.  What bounds it now is latency at 16 to 20 warps an
// SM: 16 instructions a channel forward and 31 backward fill 60% of the issue
// slots, and the warps wait for their own last instruction or for shared memory.
// A row costs a thread some 190 instructions whatever its chunks (sums across
// the group, angles, addresses).  Walking consecutive tokens with additions
// instead of divisions took more of them, and more warps per SM spill.
#include "layer_common.cuh"
#include "kernels.h"
#undef VEDA_SRC_ID
#define VEDA_SRC_ID 9   // bounds-check site id of this file (debug builds)

namespace veda {

// A channel's pair and its place in it; pair p has column p - base / 2 of its
// axis's table (base: the axis's first channel) in both pairings.
struct PairOf {
  int pair, partner;
  bool second, turned;
};
__device__ __forceinline__ PairOf pair_of(const RopeArgs& A, int ch) {
  PairOf g{0, ch, false, false};
  int base = 0;
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    const int u = ch - base, dim = A.dim[a], half = dim >> 1;
    if (u >= 0 && u < dim) {
      g.turned = true;
      g.second = A.halves ? u >= half : (u & 1);
      g.pair = (base >> 1) + (A.halves ? (g.second ? u - half : u) : u >> 1);
      g.partner = A.halves ? (g.second ? ch - half : ch + half) : ch ^ 1;
    }
    base += dim;
  }
  return g;
}

// The angles of the group's tokens in shared memory: kSlots = D + 2 rows of up
// to 64 (cos, sin).  Row r + D is fetched in iteration r over row r - 2, which
// every thread of the group has left: all of them have met at a barrier of
// iteration r - 1.
template <bool HALVES, int D>
struct Angles {
  static constexpr int kSlots = D + 2;
  static constexpr int kRow = HALVES ? 72 : 64;   // padded by one per 8 pairs where threads read with a stride
  static constexpr size_t kBytes = kSlots * kRow * sizeof(float2);
  static constexpr int kN = HALVES ? 8 : 4;       // angles per chunk
  float2* rows;
  // What this thread fetches: the pairs t and t + tpt (the second for d = 128 in one warp).
  const float2* src[2];
  int step[2], axis[2];
  bool any;
  // What it reads: bit j of `turned` for the pair of channel j (halves) or 2j, 2j + 1; and for
  // halves the pair's place, the partner's place in the warp's scratch, and whether it is the second.
  uint32_t turned;
  bool all;           // every channel of a head is turned: nothing to choose (grid-uniform)
  uint32_t at[HALVES ? 8 : 1];
  __device__ __forceinline__ static int place(int pair) { return HALVES ? pair + (pair >> 3) : pair; }
  __device__ __forceinline__ Angles(const RopeArgs& A, void* smem, const RowGroup& g, int ch0, int lph) {
    rows = static_cast<float2*>(smem) + g.group * (kSlots * kRow);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int pair = g.t + j * g.tpt;
      src[j] = nullptr;
      step[j] = axis[j] = 0;
      int base = 0;
#pragma unroll
      for (int a = 0; a < 3; ++a) {
        const int n = A.dim[a] >> 1;
        if (pair >= base && pair < base + n) {
          src[j] = A.tab[a] + (pair - base);
          step[j] = n;
          axis[j] = a;
        }
        base += n;
      }
    }
    any = src[0] != nullptr || src[1] != nullptr;
    all = A.dim[0] + A.dim[1] + A.dim[2] == A.d;
    turned = 0;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const PairOf p = pair_of(A, ch0 + (HALVES ? j : 2 * j));
      turned |= (p.turned ? 1u : 0u) << j;
      if constexpr (HALVES) {
        const int first = g.lane / lph * lph;
        at[j] = (uint32_t)place(p.pair) | (uint32_t)((first + (p.partner >> 3)) * 9 + (p.partner & 7)) << 8 |
                (p.second ? 1u << 31 : 0u);
      }
    }
  }
  __device__ __forceinline__ void fetch(const RopeArgs& A, const RowGroup& g, int slot, int n) const {
    if (!any) return;
    const int t = A.by_hw.div(n), r = n - t * A.HW, y = A.by_w.div(r), x = r - y * A.W;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (src[j] != nullptr) {
        const int pos = axis[j] == 0 ? t : axis[j] == 1 ? y : x;
        cp_async8(smem_u32(rows + slot * kRow + place(g.t + j * g.tpt)), src[j] + (long long)pos * step[j]);
      }
    }
  }
  __device__ __forceinline__ void read(int slot, int ch0, float2* cs) const {
    const float2* r = rows + slot * kRow;
    if constexpr (HALVES) {
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = r[at[j] & 0xff];
    } else {
      const float4* q = reinterpret_cast<const float4*>(r + (ch0 >> 1));
      const float4 a = q[0], b = q[1];
      cs[0] = make_float2(a.x, a.y);
      cs[1] = make_float2(a.z, a.w);
      cs[2] = make_float2(b.x, b.y);
      cs[3] = make_float2(b.z, b.w);
    }
  }
  // p turned by +angle (dir = 1) or -angle (dir = -1); a channel that is not
  // turned stays as it is, an infinity too.  `scratch`: this warp's 32 * 9
  // floats (a lane's 8 values at 9 * lane: no bank conflicts).
  __device__ __forceinline__ void apply(uint64_t* p, const float2* cs, float dir, float* scratch, int lane) const {
    if constexpr (HALVES) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) f2_split(p[k], v[2 * k], v[2 * k + 1]);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) scratch[lane * 9 + j] = v[j];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = (at[j] >> 31 ? dir : -dir) * cs[j].y;
        const float r = fmaf(v[j], cs[j].x, s * scratch[(at[j] >> 8) & 0x1ff]);
        v[j] = turned >> j & 1 ? r : v[j];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = f2(v[2 * k], v[2 * k + 1]);
    } else if (all) {
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = turn(p[j], cs[j].x, dir * cs[j].y);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (turned >> j & 1) p[j] = turn(p[j], cs[j].x, dir * cs[j].y);
      }
    }
  }
  __device__ __forceinline__ static uint64_t turn(uint64_t p, float c, float s) {
    float a, b;
    f2_split(p, a, b);
    return f2(fmaf(a, c, -b * s), fmaf(a, s, b * c));
  }
};

__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int off = lanes >> 1; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Rows in flight per group, and the warps of a CTA, which bound the registers: as
// many as leave the kernel all but a few of those it wants.
__host__ __device__ constexpr int rope_depth(int cpt) { return cpt > 2 ? 3 : 4; }
__host__ __device__ constexpr int rope_bwd_depth(int cpt) { return cpt == 4 ? 1 : 3; }
__host__ __device__ constexpr int rope_warps(int cpt) { return cpt <= 2 ? 20 : 16; }
constexpr int kRopeBwdWarps = 16;

// A token's row on its way: chunk c of it starts at (c / lph) * sh + c % lph * 8.
template <typename T, int CPT>
__device__ __forceinline__ void fetch_token(const RopeArgs& A, const Ring<T, CPT>& ring, int slot, const RowGroup& g,
                                            int nchunk, int lph, const T* row, long long sh) {
  const int shift = lph == 16 ? 4 : 3;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
#pragma unroll
    for (int j = 0; j < Ring<T, CPT>::kPieces; ++j) {
      const int c = g.t + i * g.tpt + ring.other(j);
      if (c < nchunk) ring.fetch(slot, i, j, row + (c >> shift) * sh + ((c & (lph - 1)) * 8 + ring.channel(j)));
    }
  }
}

template <typename T, int CPT, bool HALVES>
__global__ void __launch_bounds__(32 * rope_warps(CPT)) qkv_rope_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int D = rope_depth(CPT);
  __shared__ float red[kRowRed];
  extern __shared__ uint4 ring_raw[];
  const RowGroup g(A.warps);
  const Ring<T, CPT> ring(ring_raw);
  uint8_t* rest = reinterpret_cast<uint8_t*>(ring_raw) + D * Ring<T, CPT>::kBytes * blockDim.x;
  float* scratch = reinterpret_cast<float*>(rest + g.groups * Angles<HALVES, D>::kBytes) + (threadIdx.x >> 5) * (32 * 9);
  const int lph = A.d / 8, nchunk = A.heads * lph;
  const int ch0 = (g.t % lph) * 8, head0 = g.t / lph, head_step = g.tpt / lph;
  const int step = gridDim.x * g.groups, first = blockIdx.x * g.groups + g.group;
  const int slot_size = CPT * blockDim.x;
  const Angles<HALVES, D> angles(A, rest, g, ch0, lph);
  int flip = 0;
  for (int o = 0; o < A.n_order; ++o) {
    if (o > 0) __syncthreads();   // the angles' slots start over
    const int which = A.order[o];
    const int norm = which == 2 ? VEDA_NORM_NONE : A.norm;
    const T* in = static_cast<const T*>(A.in[which]);
    const long long sb = A.sb[which], sn = A.sn[which], sh = A.sh[which];
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(A.out[which]) + ch0;
    auto fetch = [&](int tok, int slot, int aslot) {
      if (tok < A.tokens) {
        const int b = A.by_n.div(tok), n = tok - b * A.N;
        if (which < 2) angles.fetch(A, g, aslot, n);
        fetch_token(A, ring, slot, g, nchunk, lph, in + b * sb + n * sn, sh);
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int s = 0; s < D; ++s) fetch(first + s * step, s * slot_size, s);
    uint64_t w[CPT][4];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = g.t + i * g.tpt;
      if (norm != VEDA_NORM_NONE && c < nchunk) load_pairs(A.w[which] + (norm == VEDA_NORM_ROW ? 8 * c : ch0), w[i]);
    }
    int slot = 0, aslot = 0;
    auto next = [](int s, int by, int n) { return s + by == n ? 0 : s + by; };
    for (int tok = first; tok < A.tokens; tok += step, flip ^= 1, slot = next(slot, slot_size, D * slot_size),
             aslot = next(aslot, 1, D + 2)) {
      uint64_t v[CPT][4];
      cp_async_wait<D - 1>();
      ring.sync();
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        to_pairs(ring.read(slot, i), v[i]);   // past the row's end: whatever is there
      }
      ring.sync();
      fetch(tok + D * step, slot, aslot >= 2 ? aslot - 2 : aslot + D);
      if (g.W == 1 || (which < 2 && norm != VEDA_NORM_ROW)) group_sync(g);   // a row's sum is a barrier itself
      if (norm != VEDA_NORM_NONE) {
        float r[CPT];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          uint64_t s2 = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) s2 = f2_fma(v[i][k], v[i][k], s2);
          r[i] = g.t + i * g.tpt < nchunk ? f2_sum(s2) : 0.f;
          ss += r[i];
        }
        if (norm == VEDA_NORM_ROW) {
          ss = rsqrtf(row_sum(g, ss, red, flip) * A.inv_n + A.eps);
#pragma unroll
          for (int i = 0; i < CPT; ++i) r[i] = ss;
        } else {
#pragma unroll
          for (int i = 0; i < CPT; ++i) r[i] = rsqrtf(head_sum(r[i], lph) * A.inv_n + A.eps);
        }
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[i][k] = f2_mul(f2_mul(v[i][k], f2_all(r[i])), w[i][k]);
        }
      }
      const int b = A.by_n.div(tok), n = tok - b * A.N;
      __nv_bfloat16* row = out + ((long long)b * A.heads * A.N + n) * A.d;
      float2 cs[Angles<HALVES, D>::kN];
      if (which < 2) angles.read(aslot, ch0, cs);
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int head = head0 + i * head_step;
        if (which < 2) angles.apply(v[i], cs, 1.f, scratch, g.lane);
        if (g.t + i * g.tpt < nchunk && VEDA_IN_BOUNDS(head < A.heads && tok < A.tokens))
          store_pairs(row + head * A.head_size, v[i], true);
      }
    }
  }
}

template <typename T, int CPT, bool HALVES>
__global__ void __launch_bounds__(32 * kRopeBwdWarps) qkv_rope_bwd_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int D = rope_bwd_depth(CPT);
  __shared__ float red[kRowRed];
  extern __shared__ uint4 ring_raw[];
  const RowGroup g(A.warps);
  const Ring<T, CPT> rx(ring_raw);
  const Ring<__nv_bfloat16, CPT> rg(ring_raw + D * Ring<T, CPT>::kBytes / 16 * blockDim.x);
  uint8_t* rest = reinterpret_cast<uint8_t*>(ring_raw) +
                  D * (Ring<T, CPT>::kBytes + Ring<__nv_bfloat16, CPT>::kBytes) * blockDim.x;
  float* scratch = reinterpret_cast<float*>(rest + g.groups * Angles<HALVES, D>::kBytes) + (threadIdx.x >> 5) * (32 * 9);
  const int lph = A.d / 8, nchunk = A.heads * lph;
  const int ch0 = (g.t % lph) * 8, head0 = g.t / lph, head_step = g.tpt / lph;
  const int step = gridDim.x * g.groups, first = blockIdx.x * g.groups + g.group;
  const int slot_size = CPT * blockDim.x;
  const Angles<HALVES, D> angles(A, rest, g, ch0, lph);
  int flip = 0;
  for (int o = 0; o < A.n_order; ++o) {
    if (o > 0) __syncthreads();   // the angles' slots start over
    const int which = A.order[o];
    const int norm = which == 2 ? VEDA_NORM_NONE : A.norm;
    const T* in = static_cast<const T*>(A.in[which]);
    const long long sb = A.sb[which], sn = A.sn[which], sh = A.sh[which];
    const __nv_bfloat16* dout = static_cast<const __nv_bfloat16*>(A.out[which]) + ch0;
    T* dx = static_cast<T*>(A.dx[which]) + ch0;
    const long long dsb = A.dsb[which], dsn = A.dsn[which], dsh = A.dsh[which];
    auto fetch = [&](int tok, int slot, int aslot) {
      if (tok < A.tokens) {
        const int b = A.by_n.div(tok), n = tok - b * A.N;
        if (which < 2) angles.fetch(A, g, aslot, n);
        const __nv_bfloat16* row = dout + ((long long)b * A.heads * A.N + n) * A.d;
#pragma unroll
        for (int i = 0; i < CPT; ++i)
          if (g.t + i * g.tpt < nchunk) rg.fetch(slot, i, 0, row + (head0 + i * head_step) * A.head_size);
        if (norm != VEDA_NORM_NONE) fetch_token(A, rx, slot, g, nchunk, lph, in + b * sb + n * sn, sh);
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int s = 0; s < D; ++s) fetch(first + s * step, s * slot_size, s);
    uint64_t w[CPT][4], acc[CPT][4];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = g.t + i * g.tpt;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = w[i][k] = 0;
      if (norm != VEDA_NORM_NONE && c < nchunk) load_pairs(A.w[which] + (norm == VEDA_NORM_ROW ? 8 * c : ch0), w[i]);
    }
    int slot = 0, aslot = 0;
    auto next = [](int s, int by, int n) { return s + by == n ? 0 : s + by; };
    for (int tok = first; tok < A.tokens; tok += step, flip ^= 1, slot = next(slot, slot_size, D * slot_size),
             aslot = next(aslot, 1, D + 2)) {
      uint64_t gv[CPT][4], v[CPT][4];
      cp_async_wait<D - 1>();
      rx.sync();
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        to_pairs(rg.read(slot, i), gv[i]);
        if (norm != VEDA_NORM_NONE) to_pairs(rx.read(slot, i), v[i]);
      }
      rx.sync();
      fetch(tok + D * step, slot, aslot >= 2 ? aslot - 2 : aslot + D);
      if (which < 2) {
        group_sync(g);
        float2 cs[Angles<HALVES, D>::kN];
        angles.read(aslot, ch0, cs);
#pragma unroll
        for (int i = 0; i < CPT; ++i) angles.apply(gv[i], cs, -1.f, scratch, g.lane);
      }
      if (norm != VEDA_NORM_NONE) {
        float s1[CPT], s2[CPT];
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          uint64_t p1 = 0, p2 = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            p1 = f2_fma(v[i][k], v[i][k], p1);
            p2 = f2_fma(f2_mul(gv[i][k], w[i][k]), v[i][k], p2);
          }
          const bool in = g.t + i * g.tpt < nchunk;   // past the row's end the ring holds anything
          s1[i] = in ? f2_sum(p1) : 0.f;
          s2[i] = in ? f2_sum(p2) : 0.f;
        }
        if (norm == VEDA_NORM_ROW) {
          float a = 0.f, c = 0.f;
#pragma unroll
          for (int i = 0; i < CPT; ++i) a += s1[i], c += s2[i];
          row_sum2(g, a, c, red, flip);
#pragma unroll
          for (int i = 0; i < CPT; ++i) s1[i] = a, s2[i] = c;
        } else {
#pragma unroll
          for (int i = 0; i < CPT; ++i) s1[i] = head_sum(s1[i], lph), s2[i] = head_sum(s2[i], lph);
        }
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const float rstd = rsqrtf(s1[i] * A.inv_n + A.eps);
          const uint64_t rr = f2_all(rstd), cc = f2_all(-s2[i] * A.inv_n * rstd * rstd);
          if (g.t + i * g.tpt >= nchunk) continue;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc[i][k] = f2_fma(f2_mul(gv[i][k], rr), v[i][k], acc[i][k]);
            gv[i][k] = f2_mul(rr, f2_fma(v[i][k], cc, f2_mul(gv[i][k], w[i][k])));
          }
        }
      }
      const int b = A.by_n.div(tok);
      T* row = dx + b * dsb + (tok - b * A.N) * dsn;
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int head = head0 + i * head_step;
        if (g.t + i * g.tpt < nchunk && VEDA_IN_BOUNDS(head < A.heads && tok < A.tokens))
          store_pairs(row + head * dsh, gv[i], A.wide);
      }
    }
    float* part = A.part[which];
    if (norm == VEDA_NORM_NONE || part == nullptr) continue;   // CTA-uniform
    // The CTA's weight gradient: one partial row per group (row norm) or per
    // run of lanes with a head's channels (head norm), over the idle ring,
    // added in order.
    const int C = norm == VEDA_NORM_ROW ? A.heads * A.d : A.d;
    const int n_rows = norm == VEDA_NORM_ROW ? g.groups : (int)blockDim.x / lph;
    float* sums = reinterpret_cast<float*>(ring_raw);
    cp_async_wait<0>();
    __syncthreads();
    if (norm == VEDA_NORM_ROW) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const int c = g.t + i * g.tpt;
        if (c < nchunk) store_shared(sums + g.group * C + 8 * c, acc[i]);
      }
    } else {
#pragma unroll
      for (int i = 1; i < CPT; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[0][k] = f2_add(acc[0][k], acc[i][k]);
      }
      store_shared(sums + (threadIdx.x / lph) * C + ch0, acc[0]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
      float s = 0.f;
      for (int k = 0; k < n_rows; ++k) s += sums[k * C + c];
      if (VEDA_IN_BOUNDS((int)blockIdx.x < A.parts)) part[(long long)blockIdx.x * C + c] = s;
    }
    __syncthreads();
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

RowSplit rope_split(int nchunk, long long tokens, int sms, bool backward) {
  // Backward three chunks a thread spill: 280 us instead of 214 at 32,760 tokens of 12 x 128.
  const int cpt = best_cpt(nchunk, backward ? 2 : 4);
  return row_split(nchunk, tokens, sms, cpt, backward ? kRopeBwdWarps : rope_warps(cpt));
}
long long rope_ctas(long long tokens, const RowSplit& r) { return (tokens + r.groups - 1) / r.groups; }

template <typename T, int CPT, bool HALVES>
cudaError_t rope_run(RopeArgs a, RowSplit r, bool backward, int sms, cudaStream_t s) {
  auto kernel = qkv_rope_kernel<T, CPT, HALVES>;
  if constexpr (CPT != 3) {
    if (backward) kernel = qkv_rope_bwd_kernel<T, CPT, HALVES>;
  }
  const size_t ring = backward ? rope_bwd_depth(CPT) * (Ring<T, CPT>::kBytes + Ring<__nv_bfloat16, CPT>::kBytes)
                               : rope_depth(CPT) * Ring<T, CPT>::kBytes;
  const size_t angles = backward ? Angles<HALVES, rope_bwd_depth(CPT)>::kBytes : Angles<HALVES, rope_depth(CPT)>::kBytes;
  const size_t group = 32 * r.W * (ring + (HALVES ? 9 * sizeof(float) : 0)) + angles;
  r.groups = std::min(r.groups, (int)(kMostSmem / group));
  r.threads = 32 * r.W * r.groups;
  const size_t smem = group * r.groups;
  static SmemLimit limits[2];
  cudaError_t e = limits[backward ? 1 : 0].allow(kernel, smem);
  if (e != cudaSuccess) return e;
  long long want = rope_ctas(a.tokens, r);
  if (backward) want = std::min(want, (long long)kBwdCtasPerSm * sms);
  const unsigned grid = resident_ctas(want, kernel, r.threads, smem, sms);
  a.parts = (int)grid;
  kernel<<<grid, r.threads, smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !backward) return e;
  SumArgs sum;
  sum.parts = a.parts;
  sum.C = a.norm == VEDA_NORM_ROW ? a.heads * a.d : a.d;
  int n = 0;
  for (int i = 0; i < 2; ++i) {
    if (a.part[i] == nullptr) continue;
    sum.part[n] = a.part[i];
    sum.out[n++] = a.dw[i];
  }
  return n == 0 ? e : launch_sum_partials(sum, n, s);
}

template <typename T>
cudaError_t rope_run(const RopeArgs& a, const RowSplit& r, bool backward, int sms, cudaStream_t s) {
  if (r.cpt == 1) return a.halves ? rope_run<T, 1, true>(a, r, backward, sms, s) : rope_run<T, 1, false>(a, r, backward, sms, s);
  if (r.cpt == 2) return a.halves ? rope_run<T, 2, true>(a, r, backward, sms, s) : rope_run<T, 2, false>(a, r, backward, sms, s);
  if (r.cpt == 3) return a.halves ? rope_run<T, 3, true>(a, r, backward, sms, s) : rope_run<T, 3, false>(a, r, backward, sms, s);
  return a.halves ? rope_run<T, 4, true>(a, r, backward, sms, s) : rope_run<T, 4, false>(a, r, backward, sms, s);
}

}  // namespace

cudaError_t launch_qkv_rope(RopeArgs a, int type, bool backward, int sms, cudaStream_t s) {
  const RowSplit r = rope_split(a.heads * a.d / 8, a.tokens, sms, backward);
  a.warps = r.W;
  a.HW = a.H * a.W;
  a.head_size = (long long)a.N * a.d;
  a.by_n = FastDiv(a.N);
  a.by_hw = FastDiv(a.HW);
  a.by_w = FastDiv(a.W);
  a.inv_n = 1.f / (float)(a.norm == VEDA_NORM_ROW ? a.heads * a.d : a.d);
  a.wide = type != VEDA_FP32 || (on_32_bytes(a.dx[0]) && on_32_bytes(a.dx[1]) && on_32_bytes(a.dx[2]));
  if (type == VEDA_BF16) return rope_run<__nv_bfloat16>(a, r, backward, sms, s);
  if (type == VEDA_FP16) return rope_run<__half>(a, r, backward, sms, s);
  return rope_run<float>(a, r, backward, sms, s);
}

// Rows of weight-gradient partials at most, each heads*d (row norm) or d (head norm) floats.
int qkv_rope_bwd_parts(long long tokens, int sms) { return (int)std::min(tokens, (long long)kBwdCtasPerSm * sms); }

cudaError_t launch_rope_table(int n, int dim, double theta, double start, double step, float* out, cudaStream_t s) {
  const long long e = (long long)n * (dim / 2);
  rope_table_kernel<<<(unsigned)((e + 255) / 256), 256, 0, s>>>(n, dim / 2, dim, log2(theta), start, step,
                                                                reinterpret_cast<float2*>(out));
  return cudaGetLastError();
}

}  // namespace veda
