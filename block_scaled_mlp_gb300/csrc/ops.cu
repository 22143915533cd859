// ops.cu - C ABI of the operators around the MLP (include/mxmlp.h): residual
// addition + RMS norm, 8-bit activation checkpoints, SwiGLU with one, ragged
// expert products.  Argument checks only; the kernels are in norm.cu, ckpt8.cu
// and ragged.cu.
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

}  // extern "C"
