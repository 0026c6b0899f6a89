// api_layers.hip -- the C-ABI entry points of the layer operators declared in
// include/gemm_f32.h: the product with its epilogue, the activation's
// gradient, layer norm and the Newton-Schulz orthogonalisation.  Argument
// checks as in api.hip: every error is a status, before anything is enqueued.
#include "gemm_f32.h"
#include "api_checks.h"
#include "launch.h"

#include <limits.h>
#include <math.h>

namespace gemmf32 {
namespace {

bool known_type(int type) { return type == GEMM_MIXED_BF16 || type == GEMM_MIXED_F16 || type == GEMM_MIXED_F32; }
bool misaligned_type(const void* p, int type) { return ((uintptr_t)p & (type == GEMM_MIXED_F32 ? 3u : 1u)) != 0; }
bool misaligned16(const void* p) { return ((uintptr_t)p & 15u) != 0; }
int64_t at_least_one(int64_t n) { return n > 1 ? n : 1; }

// Columns of the epilogue pass: 256 threads per 128 of them, below 2^32
// work-items.
constexpr int64_t kMaxPassCols = INT_MAX - 127;

// An output in place of an input: the same pointer is the same matrix only
// with the same leading dimension (or one row).
bool other_matrix(const void* out, int64_t ldo, const void* in, int64_t ldi, int64_t rows) {
    return out == in && ldo != ldi && rows > 1;
}

int check_device() {
    int dev = -1;
    return hipGetDevice(&dev) == hipSuccess && dev >= 0 ? GEMM_F32_OK : GEMM_F32_ERR_DEVICE;
}
int finish(hipError_t e) {
    if (e == hipErrorInvalidValue) return GEMM_F32_ERR_TOO_LARGE;
    return e == hipSuccess ? GEMM_F32_OK : GEMM_F32_ERR_LAUNCH;
}
int check_workspace(int64_t need, const void* workspace, int64_t bytes) {
    if (bytes < 0) return GEMM_F32_ERR_INVALID_DIM;
    if (bytes < need) return GEMM_F32_ERR_WORKSPACE;
    if (need > 0 && workspace == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (need > 0 && misaligned16(workspace)) return GEMM_F32_ERR_MISALIGNED;
    return GEMM_F32_OK;
}

// The product's checks that need no C pointer or workspace (C's leading
// dimension is given as N by the size query).
int check_linear(int op_a, int op_b, int format, int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda,
                 const uint16_t* B, int64_t ldb, int64_t ldc, const gemm_epilogue* ep) {
    if ((op_a != GEMM_F32_OP_N && op_a != GEMM_F32_OP_T) || (op_b != GEMM_F32_OP_N && op_b != GEMM_F32_OP_T))
        return GEMM_F32_ERR_INVALID_OP;
    if (format != GEMM_MIXED_BF16 && format != GEMM_MIXED_F16) return GEMM_F32_ERR_INVALID_FORMAT;
    if (ep == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (ep->c_type != format && ep->c_type != GEMM_MIXED_F32) return GEMM_F32_ERR_INVALID_TYPE;
    if (ep->bias != nullptr && ep->bias_type != format && ep->bias_type != GEMM_MIXED_F32)
        return GEMM_F32_ERR_INVALID_TYPE;
    if (ep->activation < GEMM_ACT_NONE || ep->activation > GEMM_ACT_SILU) return GEMM_F32_ERR_INVALID_ACTIVATION;
    if (ep->gradient != 0 && ep->gradient != 1) return GEMM_F32_ERR_INVALID_EPILOGUE;
    if (ep->gradient == 0 ? ep->bias_grad != nullptr : ep->bias != nullptr) return GEMM_F32_ERR_INVALID_EPILOGUE;
    if (M < 0 || N < 0 || K < 0) return GEMM_F32_ERR_INVALID_DIM;
    const int64_t a_rows = op_a ? K : M, a_cols = op_a ? M : K;
    const int64_t b_rows = op_b ? N : K, b_cols = op_b ? K : N;
    const bool reads_z = ep->gradient && ep->activation != GEMM_ACT_NONE;
    const bool uses_z = ep->gradient ? reads_z : ep->preact != nullptr;
    if (lda < at_least_one(a_cols) || ldb < at_least_one(b_cols) || ldc < at_least_one(N)) return GEMM_F32_ERR_INVALID_LD;
    if (ep->residual != nullptr && ep->ld_residual < at_least_one(N)) return GEMM_F32_ERR_INVALID_LD;
    if (uses_z && ep->ld_preact < at_least_one(N)) return GEMM_F32_ERR_INVALID_LD;
    if (N == 0) return GEMM_F32_OK;
    if (misaligned(ep->bias_grad)) return GEMM_F32_ERR_MISALIGNED;
    if (N > INT_MAX) return GEMM_F32_ERR_TOO_LARGE;
    if (M == 0) return GEMM_F32_OK;
    if ((K > 0 && (A == nullptr || B == nullptr)) || (reads_z && ep->preact == nullptr)) return GEMM_F32_ERR_NULL_PTR;
    if (K > 0 && ((((uintptr_t)A | (uintptr_t)B) & 1u) != 0)) return GEMM_F32_ERR_MISALIGNED;
    if ((ep->bias != nullptr && misaligned_type(ep->bias, ep->bias_type)) ||
        (ep->residual != nullptr && misaligned_type(ep->residual, ep->c_type)) ||
        (uses_z && misaligned_type(ep->preact, format)))
        return GEMM_F32_ERR_MISALIGNED;
    if (M > INT_MAX || K > INT_MAX) return GEMM_F32_ERR_TOO_LARGE;
    if (!extent_fits(a_rows, a_cols, lda) || !extent_fits(b_rows, b_cols, ldb) || !extent_fits(M, N, ldc) ||
        (ep->residual != nullptr && !extent_fits(M, N, ep->ld_residual)) ||
        (uses_z && !extent_fits(M, N, ep->ld_preact)))
        return GEMM_F32_ERR_TOO_LARGE;
    // at most one block of 256 threads per 64 x 64 entries: keep the grid below
    // 2^32 work-items
    const int64_t blocks64 = ((M + 63) / 64) * ((N + 63) / 64);
    if (blocks64 > (int64_t)0xFFFFFFFF / 256) return GEMM_F32_ERR_TOO_LARGE;
    return GEMM_F32_OK;
}

EpilogueArgs epilogue_args(int format, int64_t M, int64_t N, void* C, int64_t ldc, const gemm_epilogue* ep) {
    EpilogueArgs e{};
    e.M = (int)M;
    e.N = (int)N;
    e.gradient = ep->gradient;
    e.act = ep->activation;
    e.c_type = ep->c_type;
    e.C = C;
    e.ldc = ldc;
    e.bias_type = ep->bias_type;
    e.bias = ep->bias;
    e.residual = ep->residual;
    e.ldr = ep->ld_residual;
    e.z_type = format;
    e.preact = ep->preact;
    e.ldz = ep->ld_preact;
    e.bias_grad = ep->bias_grad;
    return e;
}

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
