// Launchers of the sm_100a kernels (internal to the library; the public
// surface is include/veda.h).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "veda_common.cuh"

namespace veda {

struct EstimatorWeights {
  const float* w1;
  const float* b1;
  const float* w2;
  const float* b2;
};

struct TopkArgs {
  int32_t* idx;
  float* probs;
  uint64_t timeout_ns;   // bounded-wait limit of the tensor-core estimator
  int32_t k_max;
  int32_t k_per_head[VEDA_MAX_HEADS];
};

struct AttnArgs {
  const int32_t* idx;
  int32_t k_max;
  float scale_log2;   // softmax scale * log2(e)
  void* op;           // bf16 [B, heads, NT_max*S, d] (tile-major) or [B, heads, N, d] (grid order)
  float* lse;         // fp32 [B, heads, NT_max*S] or [B, heads, N]; or null
  uint64_t timeout_ns;
  // Grid-order launches only: the heads this launch covers and, per head,
  // which of the launch's tensor maps holds its tile box.
  int32_t n_group;
  int16_t head_list[VEDA_MAX_HEADS];
  int8_t map_of_head[VEDA_MAX_HEADS];
};

// Tensor maps of one attention launch.  Tile-major operands need one map
// each; grid-order operands need one per distinct tiling (the tile box is
// part of the map), up to kMaxGridMaps per launch.
constexpr int kMaxGridMaps = 8;
template <int NM>
struct AttnMaps {
  CUtensorMap q[NM], k[NM], v[NM];
};

// Attention backward (grid order).  The dQ launch holds (Q_i, dO_i) and
// streams the selected (K, V) tiles; the dK/dV launch holds (K_j, V_j) and
// streams (Q, dO) of the Q tiles that selected j.  Maps per distinct tiling:
// a0/a1 the stationary pair, b0/b1 the moving pair.
template <int NM>
struct BwdMaps {
  CUtensorMap a0[NM], a1[NM], b0[NM], b1[NM];
};

struct BwdArgs {
  const int32_t* idx;       // [B, heads, NT_max, k_max]
  int32_t k_max;
  const int32_t* inv_off;   // [B*heads, NT_max + 1]
  const int32_t* inv_list;  // [B*heads, NT_max * k_max]
  const float2* ldt;        // [B*heads, NT_max, S]: per tile slot (L, D) = (lse log2(e), rowsum(dO * O)),
                            // (+inf, 0) on pad slots
  void* dx;                 // bf16 [B, heads, N, d]: dQ (dQ launch) or dK (dK/dV launch)
  void* dv;                 // bf16 [B, heads, N, d]: dV (dK/dV launch)
  float scale;
  float scale_log2;
  uint64_t timeout_ns;
  int32_t n_group;
  int16_t head_list[VEDA_MAX_HEADS];
  int8_t map_of_head[VEDA_MAX_HEADS];
};

struct MapArgs {
  const int32_t* rows;  // [B*heads, R]
  int32_t R;
  float scale_log2;
  float* rowmax;        // scratch [B*heads, R, NT_max, S]  (scaled, log2 domain)
  float* lse2;          // scratch [B*heads, R, S]          (log2 domain)
  float* map;           // [B, heads, R, NT_max]
  uint64_t timeout_ns;
  // Grid-order pass-1 launches only: the heads this launch covers and, per
  // head, which of the launch's tensor maps holds its tile box.
  int32_t n_group;
  int16_t head_list[VEDA_MAX_HEADS];
  int8_t map_of_head[VEDA_MAX_HEADS];
};

cudaError_t launch_permute(const Geometry& G, const void* x, void* xp, cudaStream_t s, int sms);
cudaError_t launch_unpermute(const Geometry& G, const void* xp, void* x, cudaStream_t s, int sms);
cudaError_t launch_permute_tripool(const Geometry& G, const void* x, void* xp, float* desc, cudaStream_t s);
cudaError_t launch_tripool(const Geometry& G, const void* xp, float* desc, cudaStream_t s);

size_t estimator_smem_bytes(int d, int hidden, int e);
cudaError_t launch_estimator(const Geometry& G, const float* dq, const float* dk, const EstimatorWeights& wq,
                             const EstimatorWeights& wk, int hidden, int e, float* phi, float* hid,
                             uint64_t timeout_ns, cudaStream_t s);
void score_topk_config(int ntmax, int e, int* qb, int* ntpad, size_t* smem);
// Scoring and selection.  phi: the estimator features, 2*B*heads*NT_max*e
// floats.  scores: room for the fp32 score matrix (score_matrix_bytes), or
// NULL, in which case each CTA keeps its block of scores in shared memory.
size_t score_matrix_bytes(const Geometry& G, int e);
cudaError_t launch_score_topk(const Geometry& G, const float* desc_q, const float* desc_k,
                              const EstimatorWeights& wq, const EstimatorWeights& wk, int hidden,
                              int e, float* phi, float* scores, const TopkArgs& args, cudaStream_t s);

size_t sparse_attn_smem_bytes(int d, int S, int k_max);
void sparse_attn_config(int d, int S, int k_max, int* k_stages, int* v_stages, size_t* smem);
cudaError_t launch_sparse_attn(const Geometry& G, const CUtensorMap& tq, const CUtensorMap& tk,
                               const CUtensorMap& tv, const AttnArgs& a, cudaStream_t s);
// Grid-order variant: Q/K/V tiles are fetched as 5D boxes of the grid-order
// tensors, O and the LSE are written to grid rows.  One launch covers the
// heads a.head_list[0..a.n_group); head h uses maps m.*[a.map_of_head[h]].
cudaError_t launch_sparse_attn_grid(const Geometry& G, const AttnMaps<kMaxGridMaps>& m, const AttnArgs& a,
                                    cudaStream_t s);
cudaError_t launch_tripool_grid(const Geometry& G, const void* x, float* desc, cudaStream_t s);

cudaError_t launch_tile_map(const Geometry& G, const CUtensorMap& tq, const CUtensorMap& tk,
                            const MapArgs& a, cudaStream_t s);
// Grid-order tile map: pass 1 once per group of up to kMaxGridMaps distinct
// tilings (a.head_list / a.map_of_head), then pass 2 once for all heads.
cudaError_t launch_tile_map_pass1_grid(const Geometry& G, const AttnMaps<kMaxGridMaps>& m, const MapArgs& a,
                                       cudaStream_t s);
cudaError_t launch_tile_map_pass2(const Geometry& G, const MapArgs& a, cudaStream_t s);

size_t distill_ws_bytes(const Geometry& G, int hidden, int e, int R);
cudaError_t launch_head_error(const Geometry& G, const void* o, const void* o_ref, float* err, float* ref,
                              float* part, cudaStream_t s);
cudaError_t launch_distill(const Geometry& G, const float* desc_q, const float* desc_k, const EstimatorWeights& wq,
                           const EstimatorWeights& wk, int hidden, int e, const float* map, const int32_t* rows,
                           int R, float* loss, const EstimatorWeights& gq, const EstimatorWeights& gk, void* ws,
                           uint64_t timeout_ns, cudaStream_t s);

size_t attn_bwd_ws_bytes(const Geometry& G, int k_max);
// Per tile slot (L, D) and the inverse selection lists into the workspace;
// fills a.idx, a.k_max, a.ldt, a.inv_off and a.inv_list.
cudaError_t launch_attn_bwd_prep(const Geometry& G, const void* o, const void* dout, const float* lse,
                                 const int32_t* idx, int k_max, void* ws, BwdArgs* a, cudaStream_t s);
cudaError_t launch_attn_bwd_dq(const Geometry& G, const BwdMaps<kMaxGridMaps>& m, const BwdArgs& a, cudaStream_t s);
cudaError_t launch_attn_bwd_dkdv(const Geometry& G, const BwdMaps<kMaxGridMaps>& m, const BwdArgs& a,
                                 cudaStream_t s);

// ---- operators around the attention ----

unsigned long long current_context_id();   // veda_api.cu

// n / d for 0 <= n < 2^31 by one high multiplication with a rounded-up reciprocal
// (Granlund and Montgomery, "Division by invariant integers using multiplication").
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t divisor) : d(divisor), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = (uint32_t)((((1ull << shift) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

struct NormArgs {
  long long rows;
  int C;
  const void* x;       // [rows, C], row stride ldx elements
  long long ldx;
  const void* delta;   // [rows, C], row stride ldd; or null (h = x)
  long long ldd;
  const float* w;
  float eps;
  void* h;             // [rows, C] or null
  void* y;             // [rows, C] in delta's type, or e4m3
  float* scale;        // e4m3 only: [ceil(C/128), rows]
  int warps;           // per row
  bool wide;           // fp32 outputs start on 32-byte borders
};

struct NormBwdArgs {
  long long rows;
  int C;
  const void *h, *dy, *dh;
  const float* w;
  float eps;
  void *dx, *ddelta;   // either may be null
  float* part;         // [parts, C] or null
  float* dw;
  int parts, warps;
  bool wide;           // fp32 outputs start on 32-byte borders
};

// Sums of partial rows: out[i][c] = sum_p part[i][p, c].
struct SumArgs {
  const float* part[2];
  float* out[2];
  int parts, C;
};
constexpr int kBwdCtasPerSm = 3;   // of the kernels that write partial rows

struct RopeArgs {
  int heads, d, H, W, HW, N;
  long long tokens;             // B * N, at most 2^30
  long long head_size;          // N * d
  FastDiv by_n, by_hw, by_w;
  float inv_n;                  // 1 / the channels of a norm
  int norm, halves;
  float eps;
  int dim[3];
  const float2* tab[3];
  const float* w[3];
  const void* in[3];
  void* out[3];                 // grid order: written forward, read backward
  void* dx[3];                  // backward
  long long sb[3], sn[3], sh[3], dsb[3], dsn[3], dsh[3];   // element strides of in and dx
  float* part[3];
  float* dw[2];
  int parts, warps;
  bool wide;                    // fp32 gradients start on 32-byte borders
  int order[3], n_order;        // the operands of this launch: 0 Q, 1 K, 2 V
};

struct QuantArgs {
  const void* x;
  long long rows, N;            // rows = batches * N, below 2^31
  FastDiv by_n;
  int C, d;
  long long sb, sn, sh;
  uint8_t* q;
  float* scale;
};

struct GemmArgs {
  int M, N, K, kblocks, nblocks;
  const float *sa, *sb, *bias;
  void* out;
  long long ldo;
  uint64_t timeout_ns;
  int tiles_m, tiles_n, tiles;
  int few, split;               // rows per tile of the kernel for few rows (0: the other one), CTAs per tile
  int bn;                       // columns per tile of the other one
};

cudaError_t launch_add_rms_norm(NormArgs a, int tx, int td, bool fp8, int sms, cudaStream_t s);
int add_rms_norm_bwd_parts(long long rows, int C, int sms);
cudaError_t launch_add_rms_norm_bwd(NormBwdArgs a, int tx, int td, int sms, cudaStream_t s);
cudaError_t launch_sum_partials(const SumArgs& a, int n, cudaStream_t s);

cudaError_t launch_qkv_rope(RopeArgs a, int type, bool backward, int sms, cudaStream_t s);
int qkv_rope_bwd_parts(long long tokens, int sms);
cudaError_t launch_rope_table(int n, int dim, double theta, double start, double step, float* out, cudaStream_t s);

cudaError_t launch_quant_rows(QuantArgs a, int type, cudaStream_t s);
cudaError_t launch_quant_weight(const void* w, int type, int N, int K, uint8_t* q, float* scale, cudaStream_t s);

void plan_gemm_fp8(GemmArgs* a, int sms);
cudaError_t launch_gemm_fp8(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const GemmArgs& a,
                            int out_type, int sms, cudaStream_t s);

cudaError_t launch_timeout_selftest(uint64_t timeout_ns, cudaStream_t s);
cudaError_t launch_bounds_selftest(cudaStream_t s);

}  // namespace veda
