// api_checks.h -- argument checks shared by the entry points' translation
// units (host only; not part of the public interface).
#pragma once

#include "gemm_f32.h"
#include "launch.h"

#include <limits.h>
#include <stdint.h>

namespace gemmf32 {
namespace {

inline bool misaligned(const void* ptr) { return ((uintptr_t)ptr & 3u) != 0; }

// (rows - 1) * ld + cols must be addressable with 64-bit element offsets.
inline bool extent_fits(int64_t rows, int64_t cols, int64_t ld) {
    if (rows == 0 || cols == 0) return true;
    int64_t last;
    if (__builtin_mul_overflow(rows - 1, ld, &last)) return false;
    return !__builtin_add_overflow(last, cols, &last);
}

inline bool known_type(int type) { return type == GEMM_MIXED_BF16 || type == GEMM_MIXED_F16 || type == GEMM_MIXED_F32; }
inline bool misaligned_type(const void* p, int type) { return ((uintptr_t)p & (type == GEMM_MIXED_F32 ? 3u : 1u)) != 0; }
inline bool misaligned16(const void* p) { return ((uintptr_t)p & 15u) != 0; }
inline int64_t at_least_one(int64_t n) { return n > 1 ? n : 1; }

// An output in place of an input: the same pointer is the same matrix only
// with the same leading dimension (or one row).
inline bool other_matrix(const void* out, int64_t ldo, const void* in, int64_t ldi, int64_t rows) {
    return out == in && ldo != ldi && rows > 1;
}

inline int check_device() {
    int dev = -1;
    return hipGetDevice(&dev) == hipSuccess && dev >= 0 ? GEMM_F32_OK : GEMM_F32_ERR_DEVICE;
}
inline int finish(hipError_t e) {
    if (e == hipErrorInvalidValue) return GEMM_F32_ERR_TOO_LARGE;
    return e == hipSuccess ? GEMM_F32_OK : GEMM_F32_ERR_LAUNCH;
}
inline int check_workspace(int64_t need, const void* workspace, int64_t bytes) {
    if (bytes < 0) return GEMM_F32_ERR_INVALID_DIM;
    if (bytes < need) return GEMM_F32_ERR_WORKSPACE;
    if (need > 0 && workspace == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (need > 0 && misaligned16(workspace)) return GEMM_F32_ERR_MISALIGNED;
    return GEMM_F32_OK;
}

// The product's checks that need no C pointer or workspace (C's leading
// dimension is given as N by the size query).
inline int check_linear(int op_a, int op_b, int format, int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda,
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

inline EpilogueArgs epilogue_args(int format, int64_t M, int64_t N, void* C, int64_t ldc, const gemm_epilogue* ep) {
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
