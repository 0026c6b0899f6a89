// api_layers.hip -- the C-ABI entry points of the layer operators declared in
// include/gemm_f32.h: the product with its epilogue, the activation's
// gradient, layer norm and the Newton-Schulz orthogonalisation.  Argument
// checks as in api.hip: every error is a status, before anything is enqueued.
#include "gemm_f32.h"
#include "api_checks.h"
#include "launch.h"
#include "linear_w4.h"

#include <limits.h>
#include <math.h>

namespace gemmf32 {
namespace {

// Columns of the epilogue pass: 256 threads per 128 of them, below 2^32
// work-items.
constexpr int64_t kMaxPassCols = INT_MAX - 127;

}  // namespace
}  // namespace gemmf32

using namespace gemmf32;

extern "C" int64_t gemm_mixed_epilogue_workspace_size(int op_a, int op_b, int format, int64_t M, int64_t N, int64_t K,
                                                      const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb,
                                                      const gemm_epilogue* epilogue) {
    if (check_linear(op_a, op_b, format, M, N, K, A, lda, B, ldb, at_least_one(N), epilogue) != GEMM_F32_OK) return -1;
    if (M == 0 || N == 0) return 0;
    const Gemm16Args p{(int)M, (int)N, (int)K, A, lda, B, ldb, nullptr, N};
    return linear_workspace(p, epilogue_args(format, M, N, nullptr, N, epilogue), op_a, op_b);
}

extern "C" int gemm_mixed_epilogue(int op_a, int op_b, int format, int64_t M, int64_t N, int64_t K, const uint16_t* A,
                                   int64_t lda, const uint16_t* B, int64_t ldb, void* C, int64_t ldc,
                                   const gemm_epilogue* epilogue, void* workspace, int64_t workspace_bytes,
                                   void* stream) {
    int st = check_linear(op_a, op_b, format, M, N, K, A, lda, B, ldb, ldc, epilogue);
    if (st != GEMM_F32_OK) return st;
    if (N == 0) return GEMM_F32_OK;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (M == 0) {
        if (epilogue->bias_grad == nullptr) return GEMM_F32_OK;
        if ((st = check_device()) != GEMM_F32_OK) return st;
        return finish(launch_column_sums(0, (int)N, nullptr, epilogue->bias_grad, s));
    }
    if (C == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned_type(C, epilogue->c_type)) return GEMM_F32_ERR_MISALIGNED;
    if (other_matrix(C, ldc, epilogue->residual, epilogue->ld_residual, M)) return GEMM_F32_ERR_INVALID_LD;
    const Gemm16Args p{(int)M, (int)N, (int)K, A, lda, B, ldb, nullptr, ldc};
    const EpilogueArgs e = epilogue_args(format, M, N, C, ldc, epilogue);
    st = check_workspace(linear_workspace(p, e, op_a, op_b), workspace, workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    return finish(launch_linear(p, e, s, format, op_a, op_b, workspace));
}

// ----------------------------------------- the product with a 4-bit weight

namespace {

// Blocks of 16 columns and up to 512 threads, so that a grid keeps below 2^32
// work-items with room to spare; rows by 64 in the second coordinate.
constexpr int64_t kMaxW4Cols = 1 << 25, kMaxW4Rows = 65535 * 64;

int check_w4(int format, int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const uint8_t* Q,
             int64_t ldq, int64_t group, const uint16_t* scales, int64_t ld_scales, const uint16_t* zeros,
             int64_t ld_zeros, int64_t ldc, const gemm_epilogue* ep) {
    // the checks of a 16-bit product, whose weight is not looked at
    const int st = check_linear(GEMM_F32_OP_N, GEMM_F32_OP_T, format, M, N, K, A, lda, A, at_least_one(K), ldc, ep);
    if (st != GEMM_F32_OK) return st;
    if (ep->gradient != 0) return GEMM_F32_ERR_INVALID_EPILOGUE;
    if (group != 32 && group != 64 && (group < 128 || group % 128 != 0)) return GEMM_F32_ERR_INVALID_DIM;
    if (group > INT_MAX) return GEMM_F32_ERR_TOO_LARGE;
    const int64_t bytes = K / 2 + K % 2, groups = K / group + (K % group != 0);
    if (ldq < at_least_one(bytes) || ld_scales < at_least_one(groups) ||
        (zeros != nullptr && ld_zeros < at_least_one(groups)))
        return GEMM_F32_ERR_INVALID_LD;
    if (M == 0 || N == 0) return GEMM_F32_OK;
    if (K > 0 && (Q == nullptr || scales == nullptr)) return GEMM_F32_ERR_NULL_PTR;
    if ((((uintptr_t)scales | (uintptr_t)zeros) & 1u) != 0) return GEMM_F32_ERR_MISALIGNED;
    if (!extent_fits(N, bytes, ldq) || !extent_fits(N, groups, ld_scales) ||
        (zeros != nullptr && !extent_fits(N, groups, ld_zeros)))
        return GEMM_F32_ERR_TOO_LARGE;
    if (N > kMaxW4Cols || M > kMaxW4Rows) return GEMM_F32_ERR_TOO_LARGE;
    return GEMM_F32_OK;
}

W4Args w4_args(int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const uint8_t* Q, int64_t ldq,
               int64_t group, const uint16_t* scales, int64_t ld_scales, const uint16_t* zeros, int64_t ld_zeros) {
    return W4Args{(int)M, (int)N, (int)K, A, lda, Q, ldq, (int)group, scales, ld_scales, zeros, ld_zeros};
}

}  // namespace

extern "C" int64_t gemm_w4_epilogue_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxW4Rows || N > kMaxW4Cols || K > INT_MAX) return -1;
    return M == 0 || N == 0 ? 0 : linear_w4_workspace((int)M, (int)N, (int)K);
}

extern "C" int gemm_w4_epilogue(int format, int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda,
                                const uint8_t* Q, int64_t ldq, int64_t group, const uint16_t* scales,
                                int64_t ld_scales, const uint16_t* zeros, int64_t ld_zeros, void* C, int64_t ldc,
                                const gemm_epilogue* epilogue, void* workspace, int64_t workspace_bytes,
                                void* stream) {
    int st = check_w4(format, M, N, K, A, lda, Q, ldq, group, scales, ld_scales, zeros, ld_zeros, ldc, epilogue);
    if (st != GEMM_F32_OK) return st;
    if (M == 0 || N == 0) return GEMM_F32_OK;
    if (C == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned_type(C, epilogue->c_type)) return GEMM_F32_ERR_MISALIGNED;
    if (other_matrix(C, ldc, epilogue->residual, epilogue->ld_residual, M)) return GEMM_F32_ERR_INVALID_LD;
    st = check_workspace(linear_w4_workspace((int)M, (int)N, (int)K), workspace, workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    return finish(launch_linear_w4(w4_args(M, N, K, A, lda, Q, ldq, group, scales, ld_scales, zeros, ld_zeros),
                                   epilogue_args(format, M, N, C, ldc, epilogue), reinterpret_cast<hipStream_t>(stream),
                                   format, workspace));
}

extern "C" int64_t activation_grad_workspace_size(int64_t M, int64_t N) {
    if (M < 0 || N < 0 || M > INT_MAX || N > kMaxPassCols) return -1;
    return M == 0 || N == 0 ? 0 : epilogue_pass_workspace((int)M, (int)N);
}

extern "C" int activation_grad(int activation, int format, int64_t M, int64_t N, const uint16_t* dY, int64_t ld_dy,
                               const uint16_t* preact, int64_t ld_preact, uint16_t* dZ, int64_t ld_dz,
                               float* bias_grad, void* workspace, int64_t workspace_bytes, void* stream) {
    if (format != GEMM_MIXED_BF16 && format != GEMM_MIXED_F16) return GEMM_F32_ERR_INVALID_FORMAT;
    if (activation < GEMM_ACT_NONE || activation > GEMM_ACT_SILU) return GEMM_F32_ERR_INVALID_ACTIVATION;
    if (M < 0 || N < 0) return GEMM_F32_ERR_INVALID_DIM;
    const bool reads_z = activation != GEMM_ACT_NONE;
    if (ld_dy < at_least_one(N) || (dZ != nullptr && ld_dz < at_least_one(N)) || (reads_z && ld_preact < at_least_one(N)))
        return GEMM_F32_ERR_INVALID_LD;
    if (N == 0) return GEMM_F32_OK;
    if (misaligned(bias_grad)) return GEMM_F32_ERR_MISALIGNED;
    if (M > INT_MAX || N > kMaxPassCols) return GEMM_F32_ERR_TOO_LARGE;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    int st;
    if (M == 0) {
        if (bias_grad == nullptr) return GEMM_F32_OK;
        if ((st = check_device()) != GEMM_F32_OK) return st;
        return finish(launch_column_sums(0, (int)N, nullptr, bias_grad, s));
    }
    if (dY == nullptr || (reads_z && preact == nullptr)) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned_type(dY, format) || misaligned_type(dZ, format) || (reads_z && misaligned_type(preact, format)))
        return GEMM_F32_ERR_MISALIGNED;
    if (!extent_fits(M, N, ld_dy) || (dZ != nullptr && !extent_fits(M, N, ld_dz)) ||
        (reads_z && !extent_fits(M, N, ld_preact)))
        return GEMM_F32_ERR_TOO_LARGE;
    if (other_matrix(dZ, ld_dz, dY, ld_dy, M)) return GEMM_F32_ERR_INVALID_LD;
    if (dZ == nullptr && bias_grad == nullptr) return GEMM_F32_OK;        // nothing to write
    st = check_workspace(bias_grad != nullptr ? epilogue_pass_workspace((int)M, (int)N) : 0, workspace, workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    EpilogueArgs e{};
    e.M = (int)M;
    e.N = (int)N;
    e.gradient = 1;
    e.act = activation;
    e.c_type = format;
    e.C = dZ;
    e.ldc = ld_dz;
    e.z_type = format;
    e.preact = const_cast<uint16_t*>(preact);
    e.ldz = ld_preact;
    e.bias_grad = bias_grad;
    return finish(launch_epilogue_pass(e, format, dY, ld_dy, 1, 0, static_cast<float*>(workspace), s));
}

// --------------------------------------------------------------- layer norm

namespace {

int check_norm(int type, int param_type, int64_t rows, int64_t cols, bool params) {
    if (!known_type(type) || (params && !known_type(param_type))) return GEMM_F32_ERR_INVALID_TYPE;
    if (rows < 0 || cols < 1) return GEMM_F32_ERR_INVALID_DIM;
    return GEMM_F32_OK;
}

}  // namespace

extern "C" int layer_norm(int type, int64_t rows, int64_t cols, const void* x, int64_t ldx, int param_type,
                          const void* gamma, const void* beta, float eps, void* y, int64_t ldy, float* mean,
                          float* rstd, void* stream) {
    int st = check_norm(type, param_type, rows, cols, gamma != nullptr || beta != nullptr);
    if (st != GEMM_F32_OK) return st;
    if (!(eps >= 0.0f) || !isfinite(eps)) return GEMM_F32_ERR_INVALID_SCALAR;
    if (ldx < cols || ldy < cols) return GEMM_F32_ERR_INVALID_LD;
    if (rows == 0) return GEMM_F32_OK;
    if (x == nullptr || y == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned_type(x, type) || misaligned_type(y, type) || misaligned_type(gamma, param_type) ||
        misaligned_type(beta, param_type) || misaligned(mean) || misaligned(rstd))
        return GEMM_F32_ERR_MISALIGNED;
    if (rows > INT_MAX || cols > INT_MAX || !extent_fits(rows, cols, ldx) || !extent_fits(rows, cols, ldy))
        return GEMM_F32_ERR_TOO_LARGE;
    if (other_matrix(y, ldy, x, ldx, rows)) return GEMM_F32_ERR_INVALID_LD;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    LayerNormArgs a{};
    a.rows = rows;
    a.cols = (int)cols;
    a.type = type;
    a.param_type = param_type;
    a.x = x;
    a.ldx = ldx;
    a.gamma = gamma;
    a.beta = beta;
    a.eps = eps;
    a.y = y;
    a.ldy = ldy;
    a.mean = mean;
    a.rstd = rstd;
    return finish(launch_layer_norm(a, reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int64_t layer_norm_backward_workspace_size(int type, int64_t rows, int64_t cols) {
    if (check_norm(type, 0, rows, cols, false) != GEMM_F32_OK || rows > INT_MAX || cols > INT_MAX) return -1;
    return rows == 0 ? 0 : layer_norm_backward_workspace(type, rows, (int)cols);
}

extern "C" int layer_norm_backward(int type, int64_t rows, int64_t cols, const void* dy, int64_t lddy, const void* x,
                                   int64_t ldx, const float* mean, const float* rstd, int param_type,
                                   const void* gamma, const void* residual_grad, int64_t ld_residual, void* dx,
                                   int64_t lddx, float* dgamma, float* dbeta, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    int st = check_norm(type, param_type, rows, cols, gamma != nullptr);
    if (st != GEMM_F32_OK) return st;
    if (lddy < cols || ldx < cols || lddx < cols || (residual_grad != nullptr && ld_residual < cols))
        return GEMM_F32_ERR_INVALID_LD;
    if (misaligned(dgamma) || misaligned(dbeta)) return GEMM_F32_ERR_MISALIGNED;
    if (rows > INT_MAX || cols > INT_MAX) return GEMM_F32_ERR_TOO_LARGE;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (rows == 0) {
        if (dgamma == nullptr && dbeta == nullptr) return GEMM_F32_OK;
        if ((st = check_device()) != GEMM_F32_OK) return st;
        hipError_t e = dgamma ? launch_column_sums(0, (int)cols, nullptr, dgamma, s) : hipSuccess;
        if (e == hipSuccess && dbeta) e = launch_column_sums(0, (int)cols, nullptr, dbeta, s);
        return finish(e);
    }
    if (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr)
        return GEMM_F32_ERR_NULL_PTR;
    if (misaligned_type(dy, type) || misaligned_type(x, type) || misaligned_type(dx, type) ||
        misaligned_type(residual_grad, type) || misaligned_type(gamma, param_type) || misaligned(mean) ||
        misaligned(rstd))
        return GEMM_F32_ERR_MISALIGNED;
    if (!extent_fits(rows, cols, lddy) || !extent_fits(rows, cols, ldx) || !extent_fits(rows, cols, lddx) ||
        (residual_grad != nullptr && !extent_fits(rows, cols, ld_residual)))
        return GEMM_F32_ERR_TOO_LARGE;
    if (other_matrix(dx, lddx, dy, lddy, rows) || other_matrix(dx, lddx, residual_grad, ld_residual, rows))
        return GEMM_F32_ERR_INVALID_LD;
    const bool sums = dgamma != nullptr || dbeta != nullptr;
    st = check_workspace(sums ? layer_norm_backward_workspace(type, rows, (int)cols) : 0, workspace, workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    LayerNormArgs a{};
    a.rows = rows;
    a.cols = (int)cols;
    a.type = type;
    a.param_type = param_type;
    a.x = x;
    a.ldx = ldx;
    a.gamma = gamma;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.lddy = lddy;
    a.residual_grad = residual_grad;
    a.ldr = ld_residual;
    a.dx = dx;
    a.lddx = lddx;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    return finish(launch_layer_norm_backward(a, workspace, s));
}

// ------------------------------------------------------------ Newton-Schulz

namespace {

// Checks of the sizes; batch, rows and cols each below 2^31.
int check_newton_schulz(int type, int64_t batch, int64_t rows, int64_t cols) {
    if (!known_type(type)) return GEMM_F32_ERR_INVALID_TYPE;
    if (batch < 0 || rows < 0 || cols < 0) return GEMM_F32_ERR_INVALID_DIM;
    if (batch > INT_MAX || rows > INT_MAX || cols > INT_MAX) return GEMM_F32_ERR_TOO_LARGE;
    return GEMM_F32_OK;
}

}  // namespace

extern "C" int64_t newton_schulz_workspace_size(int type, int64_t batch, int64_t rows, int64_t cols) {
    if (check_newton_schulz(type, batch, rows, cols) != GEMM_F32_OK) return -1;
    if (batch == 0 || rows == 0 || cols == 0) return 0;
    NewtonSchulzArgs a{};
    a.batch = batch;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.type = type;
    return newton_schulz_workspace(a);
}

extern "C" int newton_schulz(int type, int64_t batch, int64_t rows, int64_t cols, const void* G, int64_t ldg,
                             int64_t stride_g, int steps, float a, float b, float c, float eps, void* out, int64_t ldo,
                             int64_t stride_o, void* workspace, int64_t workspace_bytes, void* stream) {
    int st = check_newton_schulz(type, batch, rows, cols);
    if (st != GEMM_F32_OK) return st;
    if (steps < 0 || steps > 100 || !isfinite(a) || !isfinite(b) || !isfinite(c) || !(eps >= 0.0f) || !isfinite(eps))
        return GEMM_F32_ERR_INVALID_SCALAR;
    double bounds[101];
    if (!newton_schulz_bounds(steps, a, b, c, bounds)) return GEMM_F32_ERR_INVALID_SCALAR;
    if (ldg < at_least_one(cols) || ldo < at_least_one(cols) || stride_g < 0) return GEMM_F32_ERR_INVALID_LD;
    if (batch == 0 || rows == 0 || cols == 0) return GEMM_F32_OK;
    if (!extent_fits(rows, cols, ldg) || !extent_fits(rows, cols, ldo)) return GEMM_F32_ERR_TOO_LARGE;
    if (batch > 1 && stride_o < (rows - 1) * ldo + cols) return GEMM_F32_ERR_INVALID_LD;
    if (!extent_fits(batch, (rows - 1) * ldg + cols, stride_g) ||
        (batch > 1 && !extent_fits(batch, (rows - 1) * ldo + cols, stride_o)))
        return GEMM_F32_ERR_TOO_LARGE;
    if (G == nullptr || out == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned_type(G, type) || misaligned_type(out, type)) return GEMM_F32_ERR_MISALIGNED;
    NewtonSchulzArgs p{};
    p.batch = batch;
    p.rows = (int)rows;
    p.cols = (int)cols;
    p.type = type;
    p.G = G;
    p.ldg = ldg;
    p.stride_g = stride_g;
    p.out = out;
    p.ldo = ldo;
    p.stride_o = stride_o;
    p.steps = steps;
    p.a = a;
    p.b = b;
    p.c = c;
    p.eps = eps;
    p.bounds = bounds;
    const int64_t need = newton_schulz_workspace(p);
    if (need < 0) return GEMM_F32_ERR_TOO_LARGE;
    st = check_workspace(need, workspace, workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    return finish(launch_newton_schulz(p, workspace, reinterpret_cast<hipStream_t>(stream)));
}
