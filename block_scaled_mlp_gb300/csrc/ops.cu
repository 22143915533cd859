// ops.cu - C ABI of the operators around the MLP (include/mxmlp.h): residual
// addition + RMS norm, 8-bit activation checkpoints, SwiGLU with one, ragged
// expert products, routing, grouping and combining, FP8 with 128-blocks.
// Argument checks only; the kernels are in norm.cu, ckpt8.cu, ragged.cu,
// route.cu, combine.cu, fp8block.cu and fp8mm.cu.
#include <math.h>

#include "kernels.h"

using namespace mx;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Every non-null pointer of the list on a 16-byte boundary.
template <class... P>
bool all_aligned16(P... p) {
  return (aligned16(p) && ...);
}

int check_norm(int64_t M, int64_t d, bool blocks) {
  if (M < 0 || d <= 0) return fail(MX_ERR_INVALID_ARG, "norm: need M >= 0 and d > 0");
  if (d % 8 || (blocks && d % 32))
    return fail(MX_ERR_UNSUPPORTED, "norm: d must be a multiple of 8, of 32 with codes or a checkpoint (got %lld)",
                (long long)d);
  if (d > kNormMaxD) return fail(MX_ERR_UNSUPPORTED, "norm: d must be at most %lld", (long long)kNormMaxD);
  if (M > INT32_MAX - 128) return fail(MX_ERR_UNSUPPORTED, "norm: too many rows");
  return MX_OK;
}

int check_ckpt(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0) return fail(MX_ERR_INVALID_ARG, "8-bit checkpoint: need rows >= 0 and cols > 0");
  if (cols % 32) return fail(MX_ERR_UNSUPPORTED, "8-bit checkpoint: cols must be a multiple of 32 (got %lld)", (long long)cols);
  if (cols > INT32_MAX / 2 || rows > INT64_MAX / 4 / cols)
    return fail(MX_ERR_UNSUPPORTED, "8-bit checkpoint: too many elements");
  return MX_OK;
}

// Every non-null pointer of the list on a multiple of n bytes.
template <class... P>
bool aligned_to(uintptr_t n, P... p) {
  return ((reinterpret_cast<uintptr_t>(p) % n == 0) && ...);
}

// Coordinates and tile numbers are 32-bit, with room for a tile past the end.
constexpr int64_t kMaxRows = INT32_MAX - 1024;

int check_route(const void* logits, int type, int64_t T, int32_t E, int32_t k, int score, float scale) {
  if (type != MX_BF16 && type != MX_FP32) return fail(MX_ERR_INVALID_ARG, "logits must be MX_BF16 or MX_FP32");
  if (score != MX_SCORE_SOFTMAX && score != MX_SCORE_SIGMOID) return fail(MX_ERR_INVALID_ARG, "unknown score %d", score);
  if (T < 0) return fail(MX_ERR_INVALID_ARG, "T must not be negative");
  if (E < 1 || E > 1024) return fail(MX_ERR_INVALID_ARG, "E must be in [1, 1024]");
  if (k < 1 || k > 32 || k > E) return fail(MX_ERR_INVALID_ARG, "k must be in [1, 32] and at most E (got %d of %d)", k, E);
  if (!isfinite(scale)) return fail(MX_ERR_INVALID_ARG, "scale must be finite");
  if (T > kMaxRows) return fail(MX_ERR_UNSUPPORTED, "too many tokens");
  if (!aligned_to(type == MX_FP32 ? 4 : 2, logits)) return fail(MX_ERR_ALIGNMENT, "logits must be aligned to their type");
  return MX_OK;
}

int check_combine(int64_t n_rows, int64_t d, int64_t T, int32_t k) {
  if (n_rows < 0 || T < 0 || d <= 0) return fail(MX_ERR_INVALID_ARG, "combine: need rows and tokens >= 0 and d > 0");
  if (k < 1 || k > 32) return fail(MX_ERR_INVALID_ARG, "k must be in [1, 32]");
  if (d % 8) return fail(MX_ERR_UNSUPPORTED, "combine: d must be a multiple of 8 (got %lld)", (long long)d);
  if (n_rows > kMaxRows || T > kMaxRows || d > (1 << 24)) return fail(MX_ERR_UNSUPPORTED, "dimension too large");
  return MX_OK;
}

}  // namespace

extern "C" {

int mx_add_rmsnorm_fwd(const void* x, const void* residual, const void* w, int64_t M, int64_t d, float eps, void* r,
                       float* rstd, void* y, int axis, int layout, int scale_mode, void* q_row, void* s_row,
                       void* q_col, void* s_col, void* ck_codes, void* ck_scales, void* stream) {
  if (axis < 0 || axis > MX_BOTH) return fail(MX_ERR_INVALID_ARG, "axis must be 0, MX_ROW, MX_COL or MX_BOTH");
  if (axis && layout != MX_SCALE_LINEAR && layout != MX_SCALE_MMA) return fail(MX_ERR_INVALID_ARG, "unknown scale layout");
  if (axis && scale_mode != MX_SCALE_RCEIL && scale_mode != MX_SCALE_FLOOR)
    return fail(MX_ERR_INVALID_ARG, "unknown scale mode %d", scale_mode);
  if (!(eps >= 0.0f) || isinf(eps)) return fail(MX_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!ck_codes != !ck_scales) return fail(MX_ERR_INVALID_ARG, "a checkpoint needs both its codes and its scales");
  int rc = check_norm(M, d, axis || ck_codes);
  if (rc) return rc;
  if ((axis & MX_COL) && M % 32) return fail(MX_ERR_UNSUPPORTED, "columnwise codes need M %% 32 == 0 (got %lld)", (long long)M);
  if (M == 0) return MX_OK;
  if (!x || !w || !rstd || (residual && !r)) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (((axis & MX_ROW) && (!q_row || !s_row)) || ((axis & MX_COL) && (!q_col || !s_col)))
    return fail(MX_ERR_INVALID_ARG, "a requested output is null");
  if (!all_aligned16(x, residual, w, r, rstd, y, q_row, s_row, q_col, s_col, ck_codes, ck_scales))
    return fail(MX_ERR_ALIGNMENT, "norm: tensor pointers must be 16-byte aligned");
  NormFwdLaunch a{};
  a.x = x; a.residual = residual; a.w = w; a.M = M; a.d = d; a.eps = eps;
  a.r = residual ? r : nullptr; a.rstd = rstd; a.y = y; a.layout = layout;
  if (axis & MX_ROW) { a.q_row = q_row; a.s_row = s_row; }
  if (axis & MX_COL) { a.q_col = q_col; a.s_col = s_col; }
  a.ck = ck_codes; a.ck_scales = ck_scales;
  a.floor_scale = scale_mode == MX_SCALE_FLOOR;
  return launch_add_rmsnorm_fwd(a, (cudaStream_t)stream);
}

int mx_selftest_norm_clusters(int most) {
  if (most != 0 && most != 8) return fail(MX_ERR_INVALID_ARG, "most must be 0 or 8");
  set_norm_cluster_limit(most);
  return MX_OK;
}

size_t mx_add_rmsnorm_bwd_workspace(int64_t M, int64_t d) {
  if (M <= 0 || d <= 0 || d > kNormMaxD) return 0;
  return (size_t)norm_bwd_ctas(M, d) * (size_t)d * 4;
}

int mx_add_rmsnorm_bwd(const void* dy, const void* r, const void* ck_codes, const void* ck_scales, const float* rstd,
                       const void* w, const void* dres, int64_t M, int64_t d, void* dx, void* dw, void* workspace,
                       void* stream) {
  if (!ck_codes != !ck_scales) return fail(MX_ERR_INVALID_ARG, "a checkpoint needs both its codes and its scales");
  int rc = check_norm(M, d, ck_codes != nullptr);
  if (rc) return rc;
  if (!dw) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (M == 0) {
    count_launch(MX_KERNEL_MEMSET);
    return cuda_status(cudaMemsetAsync(dw, 0, (size_t)d * 2, (cudaStream_t)stream), "cudaMemsetAsync");
  }
  if (!r == !ck_codes) return fail(MX_ERR_INVALID_ARG, "pass either r or its checkpoint");
  if (!dy || !rstd || !w || !dx || !workspace) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(dy, r, ck_codes, ck_scales, rstd, w, dres, dx, dw, workspace))
    return fail(MX_ERR_ALIGNMENT, "norm: tensor pointers must be 16-byte aligned");
  NormBwdLaunch a{};
  a.dy = dy; a.r = r; a.ck = ck_codes; a.ck_scales = ck_scales; a.rstd = rstd; a.w = w; a.dres = dres;
  a.M = M; a.d = d; a.dx = dx; a.dw = dw; a.workspace = workspace;
  return launch_add_rmsnorm_bwd(a, (cudaStream_t)stream);
}

int mx_ckpt8_save(const void* x, int64_t rows, int64_t cols, void* codes, void* scales, void* stream) {
  int rc = check_ckpt(rows, cols);
  if (rc) return rc;
  if (rows == 0) return MX_OK;
  if (!x || !codes || !scales) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(x, codes, scales)) return fail(MX_ERR_ALIGNMENT, "tensor pointers must be 16-byte aligned");
  return launch_ckpt8_save(x, rows, cols, codes, scales, (cudaStream_t)stream);
}

int mx_ckpt8_load(const void* codes, const void* scales, int64_t rows, int64_t cols, void* x, void* stream) {
  int rc = check_ckpt(rows, cols);
  if (rc) return rc;
  if (rows == 0) return MX_OK;
  if (!x || !codes || !scales) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(x, codes, scales)) return fail(MX_ERR_ALIGNMENT, "tensor pointers must be 16-byte aligned");
  return launch_ckpt8_load(codes, scales, rows, cols, x, (cudaStream_t)stream);
}

int mx_swiglu_ckpt8_fwd(const void* h13, int64_t M, int64_t h, void* y, void* codes, void* scales, void* stream) {
  int rc = check_ckpt(M, h);
  if (rc) return rc;
  if (M == 0) return MX_OK;
  if (!h13 || !y || !codes || !scales) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(h13, y, codes, scales)) return fail(MX_ERR_ALIGNMENT, "tensor pointers must be 16-byte aligned");
  return launch_swiglu_ckpt8_fwd(h13, M, h, y, codes, scales, (cudaStream_t)stream);
}

int mx_swiglu_ckpt8_bwd(const void* dy, const void* codes, const void* scales, int64_t M, int64_t h, void* dh13,
                        void* y, void* stream) {
  int rc = check_ckpt(M, h);
  if (rc) return rc;
  if (M == 0) return MX_OK;
  if (!dy || !codes || !scales || !dh13) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(dy, codes, scales, dh13, y)) return fail(MX_ERR_ALIGNMENT, "tensor pointers must be 16-byte aligned");
  return launch_swiglu_ckpt8_bwd(dy, codes, scales, M, h, dh13, y, (cudaStream_t)stream);
}

int mx_ragged_mm(int mode, const void* a, const void* b, int64_t M_total, int64_t N, int64_t K, const int32_t* offs,
                 int32_t E, void* c, int32_t* err_word, void* stream) {
  if (mode < MX_RAGGED_FWD || mode > MX_RAGGED_WGRAD) return fail(MX_ERR_INVALID_ARG, "unknown ragged mode %d", mode);
  if (M_total < 0 || N <= 0 || K <= 0) return fail(MX_ERR_INVALID_ARG, "need M_total >= 0, N > 0 and K > 0");
  if (E < 1 || E > 1024) return fail(MX_ERR_INVALID_ARG, "E must be in [1, 1024]");
  if (N % 8 || K % 8)
    return fail(MX_ERR_UNSUPPORTED, "N and K must be multiples of 8 (got %lld, %lld)", (long long)N, (long long)K);
  // coordinates and tile numbers are 32-bit, with room for a tile past the end
  const int64_t most = INT32_MAX - 1024;
  if (M_total > most || N > most || K > most) return fail(MX_ERR_UNSUPPORTED, "dimension too large");
  if (!offs || (M_total > 0 && (!a || !b)) || (!c && (M_total > 0 || mode == MX_RAGGED_WGRAD)))
    return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(a, b, c)) return fail(MX_ERR_ALIGNMENT, "tensor pointers must be 16-byte aligned");
  if (M_total == 0) {
    if (mode != MX_RAGGED_WGRAD) return MX_OK;
    count_launch(MX_KERNEL_MEMSET);
    return cuda_status(cudaMemsetAsync(c, 0, (size_t)E * N * K * 2, (cudaStream_t)stream), "cudaMemsetAsync");
  }
  RaggedLaunch g{};
  g.mode = mode; g.a = a; g.b = b; g.M = M_total; g.N = N; g.K = K; g.offs = offs; g.E = E; g.c = c; g.err = err_word;
  return launch_ragged(g, (cudaStream_t)stream);
}

int mx_moe_route(const void* logits, int logits_type, int64_t T, int32_t E, int32_t k, int score, const float* bias,
                 int32_t groups, int32_t top_groups, int renorm, float scale, int32_t* ids, float* weights, void* stream) {
  int rc = check_route(logits, logits_type, T, E, k, score, scale);
  if (rc) return rc;
  if (groups < 1 || groups > 32 || E % groups)
    return fail(MX_ERR_INVALID_ARG, "groups must be in [1, 32] and divide E (got %d of %d experts)", groups, E);
  if (top_groups < 1 || top_groups > groups) return fail(MX_ERR_INVALID_ARG, "top_groups must be in [1, groups]");
  if (k > top_groups * (E / groups))
    return fail(MX_ERR_INVALID_ARG, "k = %d experts do not fit %d groups of %d", k, top_groups, E / groups);
  if (T == 0) return MX_OK;
  if (!logits || !ids || !weights) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned_to(4, bias, ids, weights)) return fail(MX_ERR_ALIGNMENT, "route: pointers must be aligned to their type");
  RouteLaunch a{};
  a.logits = logits; a.wide = logits_type == MX_FP32; a.bias = bias; a.T = T; a.E = E; a.k = k;
  a.groups = top_groups == groups ? 1 : groups;  // all of them taken: no choice
  a.top_groups = top_groups; a.score = score; a.renorm = renorm != 0; a.scale = scale; a.ids = ids; a.weights = weights;
  return launch_moe_route(a, (cudaStream_t)stream);
}

int mx_moe_route_bwd(const float* dweights, const void* logits, int logits_type, const int32_t* ids, int64_t T, int32_t E,
                     int32_t k, int score, int renorm, float scale, void* dlogits, int32_t* err_word, void* stream) {
  int rc = check_route(logits, logits_type, T, E, k, score, scale);
  if (rc) return rc;
  if (T == 0) return MX_OK;
  if (!dweights || !logits || !ids || !dlogits) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned_to(logits_type == MX_FP32 ? 4 : 2, dlogits) || !aligned_to(4, dweights, ids))
    return fail(MX_ERR_ALIGNMENT, "route: pointers must be aligned to their type");
  RouteBwdLaunch a{};
  a.dweights = dweights; a.logits = logits; a.wide = logits_type == MX_FP32; a.ids = ids; a.T = T; a.E = E; a.k = k;
  a.score = score; a.renorm = renorm != 0; a.scale = scale; a.dlogits = dlogits; a.err = err_word;
  return launch_moe_route_bwd(a, (cudaStream_t)stream);
}

size_t mx_token_group_workspace(int64_t R, int32_t E) {
  if (R <= 0 || R > kMaxRows || E < 1 || E > 1024) return 0;
  return token_group_workspace(R, E);
}

int mx_token_group(const int32_t* expert_of, int64_t R, int32_t E, int32_t* offs, int32_t* row_dst, int32_t* row_src,
                   void* workspace, int32_t* err_word, void* stream) {
  if (R < 0) return fail(MX_ERR_INVALID_ARG, "R must not be negative");
  if (E < 1 || E > 1024) return fail(MX_ERR_INVALID_ARG, "E must be in [1, 1024]");
  if (R > kMaxRows) return fail(MX_ERR_UNSUPPORTED, "too many rows");
  if (!offs || (R > 0 && (!expert_of || !row_dst || !row_src || (!workspace && token_group_workspace(R, E)))))
    return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned_to(4, expert_of, offs, row_dst, row_src) || !all_aligned16(workspace))
    return fail(MX_ERR_ALIGNMENT, "token group: pointers must be aligned to 4 bytes, the workspace to 16");
  if (R == 0) {
    count_launch(MX_KERNEL_MEMSET);
    return cuda_status(cudaMemsetAsync(offs, 0, (size_t)E * 4, (cudaStream_t)stream), "cudaMemsetAsync");
  }
  return launch_token_group(expert_of, R, E, offs, row_dst, row_src, workspace, err_word, (cudaStream_t)stream);
}

int mx_moe_combine(const void* rows, int64_t n_rows, int64_t d, const int32_t* row_dst, int64_t T, int32_t k,
                   const float* weights, const void* add, void* out, int32_t* err_word, void* stream) {
  int rc = check_combine(n_rows, d, T, k);
  if (rc) return rc;
  if (T == 0) return MX_OK;
  if ((!rows && n_rows > 0) || !row_dst || !out) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(rows, add, out) || !aligned_to(4, row_dst, weights))
    return fail(MX_ERR_ALIGNMENT, "combine: row pointers must be 16-byte aligned");
  CombineLaunch a{};
  a.rows = rows; a.n_rows = n_rows; a.d = d; a.row_dst = row_dst; a.T = T; a.k = k; a.weights = weights; a.add = add;
  a.out = out; a.err = err_word;
  return launch_moe_combine(a, (cudaStream_t)stream);
}

int mx_moe_combine_bwd(const void* dout, const void* rows, int64_t n_rows, int64_t d, const int32_t* row_dst,
                       const int32_t* row_src, int64_t T, int32_t k, const float* weights, void* drows, float* dweights,
                       int32_t* err_word, void* stream) {
  int rc = check_combine(n_rows, d, T, k);
  if (rc) return rc;
  if ((n_rows > 0 && (!rows || !row_src || !drows)) || (T > 0 && (!dout || !row_dst || !weights || !dweights)))
    return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(dout, rows, drows) || !aligned_to(4, row_dst, row_src, weights, dweights))
    return fail(MX_ERR_ALIGNMENT, "combine: row pointers must be 16-byte aligned");
  if (T == 0) {
    if (n_rows == 0) return MX_OK;
    count_launch(MX_KERNEL_MEMSET);
    return cuda_status(cudaMemsetAsync(drows, 0, (size_t)n_rows * d * 2, (cudaStream_t)stream), "cudaMemsetAsync");
  }
  CombineLaunch a{};
  a.dout = dout; a.rows = rows; a.n_rows = n_rows; a.d = d; a.row_dst = row_dst; a.row_src = row_src; a.T = T; a.k = k;
  a.weights = weights; a.drows = drows; a.dweights = dweights; a.err = err_word;
  return launch_moe_combine_bwd(a, (cudaStream_t)stream);
}

int mx_fp8_block_quantize(const void* x, int64_t rows_in, int64_t cols, const int32_t* src, int64_t rows, int32_t div,
                          void* codes, float* scales, int32_t* err_word, void* stream) {
  if (rows_in < 0 || rows < 0 || cols <= 0 || div < 1)
    return fail(MX_ERR_INVALID_ARG, "need rows >= 0, cols > 0 and div >= 1");
  if (!src && (rows != rows_in || div != 1)) return fail(MX_ERR_INVALID_ARG, "rows and div other than x's need src");
  if (cols % 16) return fail(MX_ERR_UNSUPPORTED, "cols must be a multiple of 16 (got %lld)", (long long)cols);
  if (rows_in > kMaxRows || rows > kMaxRows || cols > kMaxRows || rows * ((cols + 127) / 128) > kMaxRows * 8)
    return fail(MX_ERR_UNSUPPORTED, "dimension too large");
  if (rows == 0) return MX_OK;
  if ((!x && rows_in > 0) || !codes || !scales) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(x, codes) || !aligned_to(4, src, scales))
    return fail(MX_ERR_ALIGNMENT, "x and code buffers must be 16-byte aligned");
  return launch_fp8_block_rows(x, rows_in, cols, src, rows, div, codes, scales, err_word, (cudaStream_t)stream);
}

int mx_fp8_block_quantize_weight(const void* w, int64_t E, int64_t N, int64_t K, void* codes, void* codes_t, float* scales,
                                 void* stream) {
  if (E < 0 || N <= 0 || K <= 0) return fail(MX_ERR_INVALID_ARG, "need E >= 0, N > 0 and K > 0");
  if (N % 16 || K % 16)
    return fail(MX_ERR_UNSUPPORTED, "N and K must be multiples of 16 (got %lld, %lld)", (long long)N, (long long)K);
  if (E > 65535 || N > 65535 * 128ll || K > kMaxRows) return fail(MX_ERR_UNSUPPORTED, "dimension too large");
  if (E == 0) return MX_OK;
  if (!w || !codes || !scales) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(w, codes, codes_t) || !aligned_to(4, scales))
    return fail(MX_ERR_ALIGNMENT, "w and code buffers must be 16-byte aligned");
  return launch_fp8_block_weight(w, E, N, K, codes, codes_t, scales, (cudaStream_t)stream);
}

int mx_fp8_block_mm(int mode, const void* a, const float* sa, const void* w, const float* sw, int64_t M_total, int64_t N,
                    int64_t K, const int32_t* offs, int32_t E, void* c, int32_t* err_word, void* stream) {
  if (mode != MX_RAGGED_FWD && mode != MX_RAGGED_DGRAD) return fail(MX_ERR_INVALID_ARG, "mode must be MX_RAGGED_FWD or MX_RAGGED_DGRAD");
  if (M_total < 0 || N <= 0 || K <= 0) return fail(MX_ERR_INVALID_ARG, "need M_total >= 0, N > 0 and K > 0");
  if (E < 1 || E > 1024 || (!offs && E != 1)) return fail(MX_ERR_INVALID_ARG, "E must be in [1, 1024], 1 without offs");
  if (N % 16 || K % 16)
    return fail(MX_ERR_UNSUPPORTED, "N and K must be multiples of 16 (got %lld, %lld)", (long long)N, (long long)K);
  if (M_total > kMaxRows || N > kMaxRows || K > kMaxRows) return fail(MX_ERR_UNSUPPORTED, "dimension too large");
  if (M_total == 0) return MX_OK;
  if (!a || !sa || !w || !sw || !c) return fail(MX_ERR_INVALID_ARG, "null pointer argument");
  if (!all_aligned16(a, w, c) || !aligned_to(4, sa, sw, offs))
    return fail(MX_ERR_ALIGNMENT, "code and output pointers must be 16-byte aligned");
  Fp8MmLaunch g{};
  g.mode = mode; g.a = a; g.sa = sa; g.w = w; g.sw = sw; g.M = M_total; g.N = N; g.K = K; g.offs = offs; g.E = E; g.c = c;
  g.err = err_word;
  return launch_fp8_block_mm(g, (cudaStream_t)stream);
}

}  // extern "C"
