// C ABI of the operators around the attention: host-side validation and
// launches (declared in include/veda.h; included by veda_api.cu).

namespace veda {
namespace {

bool is_type(int t) { return t == VEDA_BF16 || t == VEDA_FP16 || t == VEDA_FP32; }

veda_status check_norm(int64_t rows, int32_t C, int x_type, int delta_type) {
  if (rows < 0 || rows > (1LL << 40)) return fail(VEDA_ERR_INVALID_ARG, "rows must be in [0, 2^40] (got %lld)", (long long)rows);
  if (C < 8 || C % 8) return fail(VEDA_ERR_INVALID_ARG, "C must be a positive multiple of 8 (got %d)", C);
  if (C > 16384) return fail(VEDA_ERR_UNSUPPORTED, "C = %d exceeds 16384 channels", C);
  if (!is_type(x_type) || !is_type(delta_type)) return fail(VEDA_ERR_INVALID_ARG, "unknown element type");
  if (x_type != delta_type && !(x_type == VEDA_FP32 && delta_type == VEDA_BF16))
    return fail(VEDA_ERR_UNSUPPORTED, "x and delta must have one type, or fp32 and bf16");
  return VEDA_OK;
}

veda_status norm_forward(const char* name, bool fp8, int64_t rows, int32_t C, int x_type, const void* x, int64_t ldx,
                         int delta_type, const void* delta, int64_t ldd, const float* weight, float eps, void* h,
                         void* y, float* scale, void* stream) {
  veda_status s = check_norm(rows, C, x_type, delta_type);
  if (s != VEDA_OK) return s;
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(VEDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (ldx < C || ldx % 8 || (delta && (ldd < C || ldd % 8)))
    return fail(VEDA_ERR_INVALID_ARG, "row strides must be multiples of 8 of at least C");
  if (rows == 0) return ok();
  if (!x || !weight || !y || (fp8 && !scale)) return fail(VEDA_ERR_INVALID_ARG, "NULL tensor argument");
  if (h == x && ldx != C) return fail(VEDA_ERR_INVALID_ARG, "h may be x only if x is dense");
  const void* ptrs[] = {x, delta, weight, h, y, scale};
  for (const void* p : ptrs)
    if (!aligned16(p)) return fail(VEDA_ERR_INVALID_ARG, "tensor arguments must be 16-byte aligned");
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.rows = rows;
  a.C = C;
  a.x = x;
  a.ldx = ldx;
  a.delta = delta;
  a.ldd = ldd;
  a.w = weight;
  a.eps = eps;
  a.h = h;
  a.y = y;
  a.scale = scale;
  const cudaError_t e = launch_add_rms_norm(a, x_type, delta_type, fp8, sm_count(), (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return ok();
}

// Validates the rotary description and fills the kernels' arguments.
veda_status make_rope(const veda_rope* r, RopeArgs* a) {
  if (r == nullptr) return fail(VEDA_ERR_INVALID_ARG, "the rope description is NULL");
  if (r->B < 1) return fail(VEDA_ERR_INVALID_ARG, "B must be >= 1 (got %d)", r->B);
  if (r->heads < 1 || r->heads > VEDA_MAX_HEADS)
    return fail(VEDA_ERR_INVALID_ARG, "heads must be in [1, %d] (got %d)", VEDA_MAX_HEADS, r->heads);
  if (r->d != 64 && r->d != 128) return fail(VEDA_ERR_UNSUPPORTED, "head dim d must be 64 or 128 (got %d)", r->d);
  if (r->grid.T < 1 || r->grid.H < 1 || r->grid.W < 1)
    return fail(VEDA_ERR_INVALID_ARG, "grid dimensions must be >= 1 (got %d x %d x %d)", r->grid.T, r->grid.H, r->grid.W);
  const long long hw = (long long)r->grid.H * r->grid.W;
  if (hw > (1LL << 30) || hw * r->grid.T > (1LL << 30)) return fail(VEDA_ERR_INVALID_ARG, "grid has too many tokens");
  const long long N = hw * r->grid.T;
  if (N * r->B > (1LL << 30)) return fail(VEDA_ERR_INVALID_ARG, "B x the grid exceeds 2^30 tokens");
  if (r->norm != VEDA_NORM_NONE && r->norm != VEDA_NORM_ROW && r->norm != VEDA_NORM_HEAD)
    return fail(VEDA_ERR_INVALID_ARG, "unknown norm %d", (int)r->norm);
  if (r->pairing != VEDA_PAIR_INTERLEAVED && r->pairing != VEDA_PAIR_HALVES)
    return fail(VEDA_ERR_INVALID_ARG, "unknown pairing %d", (int)r->pairing);
  if (!(r->eps >= 0.f) || std::isinf(r->eps)) return fail(VEDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  const int32_t dims[3] = {r->dim_t, r->dim_h, r->dim_w};
  const float* tabs[3] = {r->table_t, r->table_h, r->table_w};
  int sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (dims[i] < 0 || dims[i] > r->d || dims[i] % 2)
      return fail(VEDA_ERR_INVALID_ARG, "each axis's channels must be an even number in [0, d] (got %d)", dims[i]);
    sum += dims[i];
  }
  if (sum > r->d) return fail(VEDA_ERR_INVALID_ARG, "the axes' channels %d + %d + %d exceed d = %d", dims[0], dims[1], dims[2], r->d);
  for (int i = 0; i < 3; ++i) {
    if (dims[i] > 0 && tabs[i] == nullptr) return fail(VEDA_ERR_INVALID_ARG, "an axis with channels needs a table");
    if ((reinterpret_cast<uintptr_t>(tabs[i]) & 7u) != 0) return fail(VEDA_ERR_INVALID_ARG, "tables must be 8-byte aligned");
  }
  std::memset(a, 0, sizeof(*a));
  a->heads = r->heads;
  a->d = r->d;
  a->H = r->grid.H;
  a->W = r->grid.W;
  a->N = (int)N;
  a->tokens = N * r->B;
  a->norm = r->norm;
  a->halves = r->pairing == VEDA_PAIR_HALVES;
  a->eps = r->eps;
  for (int i = 0; i < 3; ++i) {
    a->dim[i] = dims[i];
    a->tab[i] = reinterpret_cast<const float2*>(tabs[i]);
  }
  return VEDA_OK;
}

veda_status check_tokens(const veda_tokens* t, const char* name) {
  if (t->x == nullptr) return fail(VEDA_ERR_INVALID_ARG, "%s has a NULL tensor", name);
  if (!aligned16(t->x)) return fail(VEDA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (t->stride_b < 0 || t->stride_n < 0 || t->stride_h < 0 || t->stride_b % 8 || t->stride_n % 8 || t->stride_h % 8)
    return fail(VEDA_ERR_INVALID_ARG, "the strides of %s must be multiples of 8 and not negative", name);
  return VEDA_OK;
}

size_t rope_part_bytes(const RopeArgs& a) {
  if (a.norm == VEDA_NORM_NONE) return 0;
  const bool row = a.norm == VEDA_NORM_ROW;
  const size_t C = row ? (size_t)a.heads * a.d : (size_t)a.d;
  return round256(sizeof(float) * C * qkv_rope_bwd_parts(a.tokens, sm_count()));
}

// 2D view [rows, cols] with a row stride of ld elements, boxes of box_rows rows x
// 128 bytes, 128-byte swizzle; reads past the end give zero, writes there are
// dropped.
veda_status encode_rows(CUtensorMapDataType type, int size, const void* ptr, int64_t ld, int rows, int cols,
                        int box_rows, CUtensorMap* out) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return fail(VEDA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * size};
  const cuuint32_t box[2] = {128u / size, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUresult r = fn(out, type, 2, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(VEDA_ERR_CUDA, "cuTensorMapEncodeTiled (matrix) failed (CUresult %d)", (int)r);
  return VEDA_OK;
}

}  // namespace
}  // namespace veda

extern "C" {

veda_status veda_add_rms_norm(int64_t rows, int32_t C, veda_dtype x_type, const void* x, int64_t ldx,
                              veda_dtype delta_type, const void* delta, int64_t ldd, const float* weight, float eps,
                              void* h, void* y, void* stream) {
  return norm_forward("veda_add_rms_norm", false, rows, C, x_type, x, ldx, delta_type, delta, ldd, weight, eps, h, y,
                      nullptr, stream);
}

veda_status veda_add_rms_norm_fp8(int64_t rows, int32_t C, veda_dtype x_type, const void* x, int64_t ldx,
                                  veda_dtype delta_type, const void* delta, int64_t ldd, const float* weight,
                                  float eps, void* h, void* y8, float* y_scale, void* stream) {
  return norm_forward("veda_add_rms_norm_fp8", true, rows, C, x_type, x, ldx, delta_type, delta, ldd, weight, eps, h,
                      y8, y_scale, stream);
}

veda_status veda_add_rms_norm_backward_workspace(int64_t rows, int32_t C, size_t* bytes) {
  veda_status s = check_norm(rows, C, VEDA_BF16, VEDA_BF16);
  if (s != VEDA_OK) return s;
  if (!bytes) return fail(VEDA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = rows == 0 ? 0 : round256(sizeof(float) * (size_t)C * add_rms_norm_bwd_parts(rows, C, sm_count()));
  return ok();
}

veda_status veda_add_rms_norm_backward(int64_t rows, int32_t C, veda_dtype x_type, const void* h,
                                       veda_dtype delta_type, const void* dy, const void* dh, const float* weight,
                                       float eps, void* dx, void* ddelta, float* dweight, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  veda_status s = check_norm(rows, C, x_type, delta_type);
  if (s != VEDA_OK) return s;
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(VEDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  const void* ptrs[] = {h, dy, dh, weight, dx, ddelta, dweight, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return fail(VEDA_ERR_INVALID_ARG, "tensor arguments must be 16-byte aligned");
  if (rows == 0) {
    if (dweight) {
      const cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)C, (cudaStream_t)stream);
      if (e != cudaSuccess) return cuda_fail(e, "veda_add_rms_norm_backward");
    }
    return ok();
  }
  if (!h || !dy || !weight) return fail(VEDA_ERR_INVALID_ARG, "NULL tensor argument");
  if (!dx && !ddelta && !dweight) return fail(VEDA_ERR_INVALID_ARG, "no gradient is asked for");
  if (dweight) {
    const size_t need = round256(sizeof(float) * (size_t)C * add_rms_norm_bwd_parts(rows, C, sm_count()));
    if (!workspace || workspace_bytes < need)
      return fail(VEDA_ERR_INVALID_ARG, "workspace of %zu bytes is below the %zu required", workspace ? workspace_bytes : 0, need);
  }
  NormBwdArgs a;
  std::memset(&a, 0, sizeof(a));
  a.rows = rows;
  a.C = C;
  a.h = h;
  a.dy = dy;
  a.dh = dh;
  a.w = weight;
  a.eps = eps;
  a.dx = dx;
  a.ddelta = ddelta;
  a.part = dweight ? static_cast<float*>(workspace) : nullptr;
  a.dw = dweight;
  const cudaError_t e = launch_add_rms_norm_bwd(a, x_type, delta_type, sm_count(), (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "veda_add_rms_norm_backward");
  return ok();
}

veda_status veda_quant_fp8(int32_t B, int64_t N, int32_t heads, int32_t d, veda_dtype type, const void* x,
                           int64_t stride_b, int64_t stride_n, int64_t stride_h, void* q, float* scale, void* stream) {
  if (B < 0 || N < 0) return fail(VEDA_ERR_INVALID_ARG, "B and N must be >= 0");
  if (heads < 1 || d < 8 || d % 8) return fail(VEDA_ERR_INVALID_ARG, "heads must be >= 1 and d a positive multiple of 8");
  if ((long long)heads * d > (1 << 20)) return fail(VEDA_ERR_UNSUPPORTED, "heads * d exceeds 2^20 channels");
  if (!is_type(type)) return fail(VEDA_ERR_INVALID_ARG, "unknown element type");
  if (stride_b < 0 || stride_n < 0 || stride_h < 0 || stride_b % 8 || stride_n % 8 || stride_h % 8)
    return fail(VEDA_ERR_INVALID_ARG, "strides must be multiples of 8 and not negative");
  if (B == 0 || N == 0) return ok();
  if (N >= (1LL << 31) / B) return fail(VEDA_ERR_INVALID_ARG, "B*N must be below 2^31 rows");
  if (!x || !q || !scale) return fail(VEDA_ERR_INVALID_ARG, "NULL tensor argument");
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale))
    return fail(VEDA_ERR_INVALID_ARG, "tensor arguments must be 16-byte aligned");
  QuantArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.rows = B * N;
  a.N = N;
  a.C = heads * d;
  a.d = d;
  a.sb = stride_b;
  a.sn = stride_n;
  a.sh = stride_h;
  a.q = static_cast<uint8_t*>(q);
  a.scale = scale;
  if ((a.rows + kQuantRows - 1) / kQuantRows * ((a.C + 127) / 128) >= (1LL << 31))
    return fail(VEDA_ERR_UNSUPPORTED, "too many rows and channels for one launch");
  const cudaError_t e = launch_quant_rows(a, type, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "veda_quant_fp8");
  return ok();
}

veda_status veda_quant_fp8_weight(int32_t N, int32_t K, veda_dtype type, const void* w, void* q, float* scale,
                                  void* stream) {
  if (N < 1 || K < 8 || K % 8) return fail(VEDA_ERR_INVALID_ARG, "N must be >= 1 and K a positive multiple of 8");
  if (!is_type(type)) return fail(VEDA_ERR_INVALID_ARG, "unknown element type");
  if (!w || !q || !scale) return fail(VEDA_ERR_INVALID_ARG, "NULL tensor argument");
  if (!aligned16(w) || !aligned16(q) || !aligned16(scale))
    return fail(VEDA_ERR_INVALID_ARG, "tensor arguments must be 16-byte aligned");
  if (((long long)N + 127) / 128 * (((long long)K + 127) / 128) >= (1LL << 31))
    return fail(VEDA_ERR_UNSUPPORTED, "the weight has too many blocks");
  const cudaError_t e = launch_quant_weight(w, type, N, K, static_cast<uint8_t*>(q), scale, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "veda_quant_fp8_weight");
  return ok();
}

veda_status veda_gemm_fp8(int32_t M, int32_t N, int32_t K, const void* a, int64_t lda, const float* a_scale,
                          const void* b, int64_t ldb, const float* b_scale, const float* bias, veda_dtype out_type,
                          void* out, int64_t ldo, void* stream) {
  if (M < 0 || N < 8 || N % 8) return fail(VEDA_ERR_INVALID_ARG, "M must be >= 0 and N a positive multiple of 8 (got %d, %d)", M, N);
  if (K < 16 || K % 16) return fail(VEDA_ERR_INVALID_ARG, "K must be a positive multiple of 16 (got %d)", K);
  if (M > (1 << 30) || N > (1 << 30) || K > (1 << 30)) return fail(VEDA_ERR_UNSUPPORTED, "M, N and K must be at most 2^30");
  if (lda < K || lda % 16 || ldb < K || ldb % 16 || lda > (1LL << 39) || ldb > (1LL << 39))
    return fail(VEDA_ERR_INVALID_ARG, "lda and ldb must be multiples of 16 of at least K");
  if (ldo < N || ldo % 8 || ldo > (1LL << 37)) return fail(VEDA_ERR_INVALID_ARG, "ldo must be a multiple of 8 of at least N");
  if (out_type != VEDA_BF16 && out_type != VEDA_FP32) return fail(VEDA_ERR_UNSUPPORTED, "out must be bf16 or fp32");
  if (M == 0) return ok();
  if (!a || !a_scale || !b || !b_scale || !out) return fail(VEDA_ERR_INVALID_ARG, "NULL tensor argument");
  const void* ptrs[] = {a, a_scale, b, b_scale, bias, out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return fail(VEDA_ERR_INVALID_ARG, "tensor arguments must be 16-byte aligned");
  if (((long long)M + 127) / 128 * (((long long)N + 127) / 128) >= (1LL << 30))
    return fail(VEDA_ERR_UNSUPPORTED, "the product has too many tiles");
  GemmArgs g;
  std::memset(&g, 0, sizeof(g));
  g.M = M;
  g.N = N;
  g.K = K;
  g.kblocks = (K + 127) / 128;
  g.nblocks = (N + 127) / 128;
  g.sa = a_scale;
  g.sb = b_scale;
  g.bias = bias;
  g.out = out;
  g.ldo = ldo;
  g.timeout_ns = g_timeout_ns;
  const int sms = sm_count();
  plan_gemm_fp8(&g, sms);
  CUtensorMap ta, tb, tc;
  veda_status s;
  const bool wide = out_type == VEDA_FP32;
  if ((s = encode_rows(CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a, lda, M, K, g.few ? g.few : 128, &ta)) != VEDA_OK ||
      (s = encode_rows(CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, b, ldb, N, K, g.few ? 128 : g.bn / 2, &tb)) != VEDA_OK ||
      (s = encode_rows(wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, wide ? 4 : 2, out, ldo,
                       M, N, 32, &tc)) != VEDA_OK)
    return s;
  const cudaError_t e = launch_gemm_fp8(ta, tb, tc, g, out_type, sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "veda_gemm_fp8");
  return ok();
}

veda_status veda_rope_table(int32_t n, int32_t dim, double theta, double start, double step, float* table,
                            void* stream) {
  if (n < 0) return fail(VEDA_ERR_INVALID_ARG, "n must be >= 0 (got %d)", n);
  if (dim < 2 || dim > 128 || dim % 2) return fail(VEDA_ERR_INVALID_ARG, "dim must be even in [2, 128] (got %d)", dim);
  if (!(theta > 0) || std::isinf(theta) || !std::isfinite(start) || !std::isfinite(step))
    return fail(VEDA_ERR_INVALID_ARG, "theta must be positive, start and step finite");
  if (n == 0) return ok();
  if (!table) return fail(VEDA_ERR_INVALID_ARG, "table is NULL");
  if ((reinterpret_cast<uintptr_t>(table) & 7u) != 0) return fail(VEDA_ERR_INVALID_ARG, "table must be 8-byte aligned");
  const cudaError_t e = launch_rope_table(n, dim, theta, start, step, table, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "veda_rope_table");
  return ok();
}

veda_status veda_qkv_norm_rope(const veda_rope* r, veda_dtype type, const veda_tokens* q, const veda_tokens* k,
                               const veda_tokens* v, const float* wq, const float* wk, void* q_out, void* k_out,
                               void* v_out, void* stream) {
  RopeArgs a;
  veda_status s = make_rope(r, &a);
  if (s != VEDA_OK) return s;
  if (!is_type(type)) return fail(VEDA_ERR_INVALID_ARG, "unknown element type");
  const veda_tokens* in[3] = {q, k, v};
  void* out[3] = {q_out, k_out, v_out};
  const float* w[3] = {wq, wk, nullptr};
  const char* names[3] = {"q", "k", "v"};
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    if ((in[i] == nullptr) != (out[i] == nullptr))
      return fail(VEDA_ERR_INVALID_ARG, "%s and its output must be given together", names[i]);
    if (in[i] == nullptr) continue;
    if ((s = check_tokens(in[i], names[i])) != VEDA_OK) return s;
    if (!aligned16(out[i])) return fail(VEDA_ERR_INVALID_ARG, "outputs must be 16-byte aligned");
    if (i < 2 && a.norm != VEDA_NORM_NONE && (!w[i] || !aligned16(w[i])))
      return fail(VEDA_ERR_INVALID_ARG, "the norm of %s needs a 16-byte aligned weight", names[i]);
    a.in[i] = in[i]->x;
    a.out[i] = out[i];
    a.w[i] = w[i];
    a.sb[i] = in[i]->stride_b;
    a.sn[i] = in[i]->stride_n;
    a.sh[i] = in[i]->stride_h;
    a.order[n++] = i;
  }
  if (n == 0) return fail(VEDA_ERR_INVALID_ARG, "no operand is given");
  a.n_order = n;
  const cudaError_t e = launch_qkv_rope(a, type, false, sm_count(), (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "veda_qkv_norm_rope");
  return ok();
}

veda_status veda_qkv_norm_rope_backward_workspace(const veda_rope* r, size_t* bytes) {
  RopeArgs a;
  veda_status s = make_rope(r, &a);
  if (s != VEDA_OK) return s;
  if (!bytes) return fail(VEDA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 2 * rope_part_bytes(a);
  return ok();
}

veda_status veda_qkv_norm_rope_backward(const veda_rope* r, veda_dtype type, const veda_tokens* q,
                                        const veda_tokens* k, const float* wq, const float* wk, const void* d_q,
                                        const void* d_k, const void* d_v, const veda_tokens* dq,
                                        const veda_tokens* dk, const veda_tokens* dv, float* dwq, float* dwk,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  RopeArgs a;
  veda_status s = make_rope(r, &a);
  if (s != VEDA_OK) return s;
  if (!is_type(type)) return fail(VEDA_ERR_INVALID_ARG, "unknown element type");
  const veda_tokens* in[3] = {q, k, nullptr};
  const void* dout[3] = {d_q, d_k, d_v};
  const veda_tokens* dx[3] = {dq, dk, dv};
  const float* w[3] = {wq, wk, nullptr};
  float* dw[3] = {dwq, dwk, nullptr};
  const char* names[3] = {"q", "k", "v"};
  const size_t part = rope_part_bytes(a);
  bool needs_part = false;
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    if ((dout[i] == nullptr) != (dx[i] == nullptr))
      return fail(VEDA_ERR_INVALID_ARG, "the gradients of %s and of its output must be given together", names[i]);
    if (dw[i] != nullptr && (dout[i] == nullptr || a.norm == VEDA_NORM_NONE))
      return fail(VEDA_ERR_INVALID_ARG, "a weight gradient of %s needs its upstream gradient and a norm", names[i]);
    if (dout[i] == nullptr) continue;
    if (!aligned16(dout[i])) return fail(VEDA_ERR_INVALID_ARG, "tensor arguments must be 16-byte aligned");
    if ((s = check_tokens(dx[i], names[i])) != VEDA_OK) return s;
    if ((a.heads > 1 && dx[i]->stride_h < a.d) || (a.N > 1 && dx[i]->stride_n < a.d) || (r->B > 1 && dx[i]->stride_b < a.d))
      return fail(VEDA_ERR_INVALID_ARG, "the gradient of %s has overlapping rows", names[i]);
    if (i < 2 && a.norm != VEDA_NORM_NONE) {
      if (!in[i]) return fail(VEDA_ERR_INVALID_ARG, "the norm's backward needs %s", names[i]);
      if ((s = check_tokens(in[i], names[i])) != VEDA_OK) return s;
      if (!w[i] || !aligned16(w[i]) || !aligned16(dw[i]))
        return fail(VEDA_ERR_INVALID_ARG, "the weight and weight gradient of %s must be given and 16-byte aligned", names[i]);
      a.in[i] = in[i]->x;
      a.sb[i] = in[i]->stride_b;
      a.sn[i] = in[i]->stride_n;
      a.sh[i] = in[i]->stride_h;
      a.w[i] = w[i];
      if (dw[i]) {
        a.part[i] = reinterpret_cast<float*>(static_cast<char*>(workspace) + (i ? part : 0));
        a.dw[i] = dw[i];
        needs_part = true;
      }
    }
    a.out[i] = const_cast<void*>(dout[i]);   // read only
    a.dx[i] = dx[i]->x;
    a.dsb[i] = dx[i]->stride_b;
    a.dsn[i] = dx[i]->stride_n;
    a.dsh[i] = dx[i]->stride_h;
    a.order[n++] = i;
  }
  if (n == 0) return fail(VEDA_ERR_INVALID_ARG, "no upstream gradient is given");
  if (needs_part && (!workspace || !aligned16(workspace) || workspace_bytes < 2 * part))
    return fail(VEDA_ERR_INVALID_ARG, "workspace of %zu bytes, 16-byte aligned, is needed (got %zu)", 2 * part,
                workspace ? workspace_bytes : 0);
  a.n_order = n;
  const cudaError_t e = launch_qkv_rope(a, type, true, sm_count(), (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "veda_qkv_norm_rope_backward");
  return ok();
}

}  // extern "C"
