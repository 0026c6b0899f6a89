// api_grouped.hip -- the C-ABI entry points of the layer whose rows belong to
// groups with a weight each.  Argument checks as in api.hip: every error is a
// status, before anything is enqueued.
#include "gemm_f32.h"
#include "api_checks.h"
#include "grouped_kernels.h"

namespace gemmf32 {
namespace {

// Blocks of the groups' sums are a grid's second coordinate.
constexpr int64_t kMaxGroups = 65535;

int check_groups(int64_t groups, const int32_t* offsets) {
    if (groups < 0) return GEMM_F32_ERR_INVALID_DIM;
    if (groups > kMaxGroups) return GEMM_F32_ERR_TOO_LARGE;
    if (groups > 0 && offsets == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned(offsets)) return GEMM_F32_ERR_MISALIGNED;
    return GEMM_F32_OK;
}

// The last group's matrix has to be addressable, as its elements are.
bool groups_fit(int64_t groups, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
    return extent_fits(rows, cols, ld) && (rows == 0 || extent_fits(groups, (rows - 1) * ld + cols, stride));
}

int check_grouped(int op_b, int format, int64_t groups, int64_t M, int64_t N, int64_t K, const uint16_t* A,
                  int64_t lda, const uint16_t* B, int64_t ldb, int64_t stride_b, const int32_t* offsets, int64_t ldc,
                  const gemm_epilogue* ep, int64_t ld_bias) {
    int st = check_groups(groups, offsets);
    if (st != GEMM_F32_OK) return st;
    // without groups there is no weight: its pointer is not looked at
    st = check_linear(GEMM_F32_OP_N, op_b, format, M, N, K, A, lda, groups > 0 ? B : A, ldb, ldc, ep);
    if (st != GEMM_F32_OK) return st;
    if (ep->gradient != 0) return GEMM_F32_ERR_INVALID_EPILOGUE;
    if (stride_b < 0 || (ep->bias != nullptr && ld_bias < 0)) return GEMM_F32_ERR_INVALID_LD;
    if (M == 0 || N == 0) return GEMM_F32_OK;
    if (!groups_fit(groups, op_b ? N : K, op_b ? K : N, ldb, stride_b) ||
        (ep->bias != nullptr && !extent_fits(groups, N, ld_bias)))
        return GEMM_F32_ERR_TOO_LARGE;
    // a block of 256 threads per tile: the grid below 2^32 work-items
    if (grouped_row_tiles(M, groups, kGroupedSmallTile) * ((N + kGroupedSmallTile - 1) / kGroupedSmallTile) >
        (int64_t)0x7FFFFFFF / 256)
        return GEMM_F32_ERR_TOO_LARGE;
    return GEMM_F32_OK;
}

int check_grouped_grad(int format, int64_t groups, int64_t rows, int64_t M, int64_t N, const uint16_t* A, int64_t lda,
                       const uint16_t* B, int64_t ldb, const int32_t* offsets, int c_type, int64_t ldc,
                       int64_t stride_c) {
    if (format != GEMM_MIXED_BF16 && format != GEMM_MIXED_F16) return GEMM_F32_ERR_INVALID_FORMAT;
    if (c_type != format && c_type != GEMM_MIXED_F32) return GEMM_F32_ERR_INVALID_TYPE;
    if (rows < 0 || M < 0 || N < 0) return GEMM_F32_ERR_INVALID_DIM;
    const int st = check_groups(groups, offsets);
    if (st != GEMM_F32_OK) return st;
    if (lda < at_least_one(M) || ldb < at_least_one(N) || ldc < at_least_one(N)) return GEMM_F32_ERR_INVALID_LD;
    if (M == 0 || N == 0 || groups == 0) return GEMM_F32_OK;
    if (rows > INT_MAX || M > INT_MAX || N > INT_MAX || !extent_fits(rows, M, lda) || !extent_fits(rows, N, ldb) ||
        !extent_fits(M, N, ldc))
        return GEMM_F32_ERR_TOO_LARGE;
    if (groups > 1 && stride_c < (M - 1) * ldc + N) return GEMM_F32_ERR_INVALID_LD;
    if (groups > 1 && !groups_fit(groups, M, N, ldc, stride_c)) return GEMM_F32_ERR_TOO_LARGE;
    const int64_t tiles = ((M + kGroupedSmallTile - 1) / kGroupedSmallTile) * ((N + kGroupedSmallTile - 1) / kGroupedSmallTile);
    if (tiles > (int64_t)0x7FFFFFFF / 256 || tiles * groups > (int64_t)0x7FFFFFFF / 256) return GEMM_F32_ERR_TOO_LARGE;
    if (rows > 0 && (A == nullptr || B == nullptr)) return GEMM_F32_ERR_NULL_PTR;
    if (rows > 0 && ((((uintptr_t)A | (uintptr_t)B) & 1u) != 0)) return GEMM_F32_ERR_MISALIGNED;
    return GEMM_F32_OK;
}

Gemm16Args product(int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb) {
    return Gemm16Args{(int)M, (int)N, (int)K, A, lda, B, ldb, nullptr, 0};
}

// The epilogue of the weights' gradient: the sums as they are.
EpilogueArgs plain_epilogue(int64_t M, int64_t N, int c_type, void* C, int64_t ldc) {
    EpilogueArgs e{};
    e.M = (int)M;
    e.N = (int)N;
    e.c_type = c_type;
    e.C = C;
    e.ldc = ldc;
    return e;
}

}  // namespace
}  // namespace gemmf32

using namespace gemmf32;

extern "C" int64_t gemm_mixed_grouped_workspace_size(int op_b, int format, int64_t groups, int64_t M, int64_t N,
                                                     int64_t K, const uint16_t* A, int64_t lda, const uint16_t* B,
                                                     int64_t ldb, int64_t stride_b, const int32_t* offsets,
                                                     const gemm_epilogue* epilogue, int64_t ld_bias) {
    if (check_grouped(op_b, format, groups, M, N, K, A, lda, B, ldb, stride_b, offsets, at_least_one(N), epilogue,
                      ld_bias) != GEMM_F32_OK)
        return -1;
    if (groups == 0 || M == 0 || N == 0) return 0;
    const GroupedArgs g{(int)groups, offsets, (int)M, stride_b, ld_bias};
    return grouped_workspace(g, product(M, N, K, A, lda, B, ldb), op_b);
}

extern "C" int gemm_mixed_grouped(int op_b, int format, int64_t groups, int64_t M, int64_t N, int64_t K,
                                  const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb, int64_t stride_b,
                                  const int32_t* offsets, void* C, int64_t ldc, const gemm_epilogue* epilogue,
                                  int64_t ld_bias, void* workspace, int64_t workspace_bytes, void* stream) {
    int st = check_grouped(op_b, format, groups, M, N, K, A, lda, B, ldb, stride_b, offsets, ldc, epilogue, ld_bias);
    if (st != GEMM_F32_OK) return st;
    if (groups == 0 || M == 0 || N == 0) return GEMM_F32_OK;
    if (C == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned_type(C, epilogue->c_type)) return GEMM_F32_ERR_MISALIGNED;
    if (other_matrix(C, ldc, epilogue->residual, epilogue->ld_residual, M)) return GEMM_F32_ERR_INVALID_LD;
    const GroupedArgs g{(int)groups, offsets, (int)M, stride_b, ld_bias};
    const Gemm16Args p = product(M, N, K, A, lda, B, ldb);
    const EpilogueArgs e = epilogue_args(format, M, N, C, ldc, epilogue);
    st = check_workspace(grouped_workspace(g, p, op_b), workspace, workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    return finish(launch_grouped(g, p, e, reinterpret_cast<hipStream_t>(stream), format, op_b, workspace));
}

extern "C" int64_t gemm_mixed_grouped_grad_workspace_size(int format, int64_t groups, int64_t rows, int64_t M,
                                                          int64_t N, const uint16_t* A, int64_t lda, const uint16_t* B,
                                                          int64_t ldb, const int32_t* offsets, int c_type) {
    // larger sizes are refused before the stride is looked at
    const int64_t stride_c = M > INT_MAX || N > INT_MAX ? 0 : at_least_one(M) * at_least_one(N);
    if (check_grouped_grad(format, groups, rows, M, N, A, lda, B, ldb, offsets, c_type, at_least_one(N), stride_c) !=
        GEMM_F32_OK)
        return -1;
    if (groups == 0 || M == 0 || N == 0) return 0;
    const GroupedArgs g{(int)groups, offsets, (int)rows, M * N, 0};
    return grouped_grad_workspace(g, product(M, N, 0, A, lda, B, ldb));
}

extern "C" int gemm_mixed_grouped_grad(int format, int64_t groups, int64_t rows, int64_t M, int64_t N,
                                       const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb,
                                       const int32_t* offsets, int c_type, void* C, int64_t ldc, int64_t stride_c,
                                       void* workspace, int64_t workspace_bytes, void* stream) {
    int st = check_grouped_grad(format, groups, rows, M, N, A, lda, B, ldb, offsets, c_type, ldc, stride_c);
    if (st != GEMM_F32_OK) return st;
    if (groups == 0 || M == 0 || N == 0) return GEMM_F32_OK;
    if (C == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned_type(C, c_type)) return GEMM_F32_ERR_MISALIGNED;
    const GroupedArgs g{(int)groups, offsets, (int)rows, stride_c, 0};
    const Gemm16Args p = product(M, N, 0, A, lda, B, ldb);
    const EpilogueArgs e = plain_epilogue(M, N, c_type, C, ldc);
    st = check_workspace(grouped_grad_workspace(g, p), workspace, workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    return finish(launch_grouped_grad(g, p, e, reinterpret_cast<hipStream_t>(stream), format, workspace));
}

extern "C" int64_t activation_grad_grouped_workspace_size(int64_t groups, int64_t M, int64_t N) {
    if (groups < 0 || groups > kMaxGroups || M < 0 || N < 0 || M > INT_MAX || N > INT_MAX) return -1;
    return N == 0 || groups == 0 ? 0 : grouped_activation_workspace(M, groups, N);
}

extern "C" int activation_grad_grouped(int activation, int format, int64_t groups, int64_t M, int64_t N,
                                       const uint16_t* dY, int64_t ld_dy, const uint16_t* preact, int64_t ld_preact,
                                       const int32_t* offsets, uint16_t* dZ, int64_t ld_dz, float* bias_grad,
                                       void* workspace, int64_t workspace_bytes, void* stream) {
    if (format != GEMM_MIXED_BF16 && format != GEMM_MIXED_F16) return GEMM_F32_ERR_INVALID_FORMAT;
    if (activation < GEMM_ACT_NONE || activation > GEMM_ACT_SILU) return GEMM_F32_ERR_INVALID_ACTIVATION;
    if (M < 0 || N < 0) return GEMM_F32_ERR_INVALID_DIM;
    int st = check_groups(groups, offsets);
    if (st != GEMM_F32_OK) return st;
    const bool reads_z = activation != GEMM_ACT_NONE;
    if (ld_dy < at_least_one(N) || (dZ != nullptr && ld_dz < at_least_one(N)) || (reads_z && ld_preact < at_least_one(N)))
        return GEMM_F32_ERR_INVALID_LD;
    if (N == 0 || groups == 0) return GEMM_F32_OK;
    if (misaligned(bias_grad)) return GEMM_F32_ERR_MISALIGNED;
    if (M > INT_MAX || N > INT_MAX) return GEMM_F32_ERR_TOO_LARGE;
    if (M > 0) {
        if (dY == nullptr || (reads_z && preact == nullptr)) return GEMM_F32_ERR_NULL_PTR;
        if (misaligned_type(dY, format) || misaligned_type(dZ, format) || (reads_z && misaligned_type(preact, format)))
            return GEMM_F32_ERR_MISALIGNED;
        if (!extent_fits(M, N, ld_dy) || (dZ != nullptr && !extent_fits(M, N, ld_dz)) ||
            (reads_z && !extent_fits(M, N, ld_preact)))
            return GEMM_F32_ERR_TOO_LARGE;
        if (other_matrix(dZ, ld_dz, dY, ld_dy, M)) return GEMM_F32_ERR_INVALID_LD;
    }
    if ((dZ == nullptr || M == 0) && bias_grad == nullptr) return GEMM_F32_OK;        // nothing to write
    st = check_workspace(bias_grad != nullptr ? grouped_activation_workspace(M, groups, N) : 0, workspace,
                         workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    const GroupedArgs g{(int)groups, offsets, (int)M, 0, 0};
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
    return finish(launch_grouped_activation(g, e, dY, ld_dy, static_cast<float*>(workspace),
                                            reinterpret_cast<hipStream_t>(stream)));
}
