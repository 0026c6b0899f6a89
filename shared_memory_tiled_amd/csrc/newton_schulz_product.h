// newton_schulz_product.h -- one product of a Newton-Schulz step: its
// description and what happens to its entries (shared by the kernels on large
// and on small tiles; not part of the public interface).
//
// Matrices are kept as two planes of binary16 values, high and low, whose sum
// times a power of two is the entry (22 bits; `plane` elements apart).  Sizes
// are padded to multiples of 64 with zeros, which the steps keep.  The two
// symmetric matrices are kept without their diagonal, which is a binary32
// vector of its own: near the end it is the large part of them, and the
// off-diagonal entries' rounding matters the less.
//
//   kGram    D + S = X X^T (or X^T X)           S: zero diagonal
//   kPoly    E + T = b (D + S) + c (D + S)^2, the product being S S:
//            (D + S)^2 = S S + (d_i + d_j) S_ij + d_i^2 on the diagonal
//   kUpdate, kUpdateColumns   X <- (a + e) X + T X, e of the row;
//            X <- X (a + e) + X T, e of the column
#pragma once

#include "mfma16_common.h"

namespace gemmf32 {

enum { kGram = 0, kPoly = 1, kUpdate = 2, kUpdateColumns = 3 };

struct NsProduct {
    int M, N, K, batch;                       // padded sizes of the product
    int stage;                                // kGram, kPoly, kUpdate, kUpdateColumns
    int terms;                                // 1: high planes only, 3: see WideCore
    const uint16_t* A; int64_t lda, plane_a, stride_a;      // factors (stride: from matrix to matrix)
    const uint16_t* B; int64_t ldb, plane_b, stride_b;
    float unscale;                            // product of the factors' scales
    const uint16_t* in; int64_t ldi, plane_i, stride_i;     // kPoly: S; updates: X
    float in_unscale;
    const float* diag_in; float* diag_out;    // one vector of diag_n per matrix
    int diag_n;
    float a, b, c;
    uint16_t* out; int64_t ldo, plane_o, stride_o;          // planes, or (final_out) the caller's matrix
    float out_scale;
    void* final_out; int final_type; int64_t final_ld, final_stride;
    int rows, cols;                           // of final_out
};

// Tiles of 256, 192 or 160 (newton_schulz_wide.hip), and of 128 or 64 with K
// split over the waves (newton_schulz_ksplit128.hip, newton_schulz_ksplit.hip).  op_a: kGram of X^T X (the stage
// says the rest of how the factors are stored).
hipError_t launch_ns_wide(const NsProduct& p, int bt, int op_a, hipStream_t s);
hipError_t launch_ns_ksplit128(const NsProduct& p, int op_a, hipStream_t s);
hipError_t launch_ns_ksplit(const NsProduct& p, int op_a, hipStream_t s);

#ifdef __HIPCC__
namespace {

typedef _Float16 half_t;

// Element `index` of a plane whose base is the same for every lane: planes
// are below 2^31 bytes (newton_schulz_workspace), so the place is a 32-bit
// offset; rows and leading dimensions are below 2^24.
template <typename T>
__device__ __forceinline__ T* plane_at(T* base, uint32_t index) {
    using C = std::conditional_t<std::is_const_v<T>, const char, char>;
    return reinterpret_cast<T*>(reinterpret_cast<C*>(base) + 2 * index);
}
__device__ __forceinline__ uint32_t plane_index(int row, int64_t ld, int col) {
    return __umul24((unsigned)row, (unsigned)ld) + (unsigned)col;
}

// W consecutive plane values as loaded, and their value over the scale.
template <int W, bool LOW>
struct PlaneRun {
    half_t h[W], l[LOW ? W : 1];
    __device__ __forceinline__ void load(const uint16_t* base, uint32_t index, int64_t plane) {
        __builtin_memcpy(h, plane_at(base, index), sizeof(h));
        if constexpr (LOW) __builtin_memcpy(l, plane_at(base + plane, index), sizeof(l));
    }
    __device__ __forceinline__ float value(int e) const { return LOW ? (float)h[e] + (float)l[e] : (float)h[e]; }
};
// The plane, or both planes, of W scaled values.
template <int W, bool LOW>
__device__ __forceinline__ void store_planes(uint16_t* base, uint32_t index, int64_t plane, const float (&v)[W]) {
    half_t h[W], l[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
        h[e] = (half_t)v[e];
        l[e] = (half_t)(v[e] - (float)h[e]);
    }
    __builtin_memcpy(plane_at(base, index), h, sizeof(h));
    if constexpr (LOW) __builtin_memcpy(plane_at(base + plane, index), l, sizeof(l));
}

// A run of W columns: what it reads of S or X, and the epilogue.  S and T
// have a low plane with TERMS = 3 only (without it S's rounding meets T's
// own, of the same 11 bits).
template <int STAGE, int TERMS, int W>
struct NsRun {
    static constexpr bool LOW = STAGE >= kUpdate || TERMS == 3;      // of the matrix read and of the one stored
    PlaneRun<W, LOW> in;
    __device__ __forceinline__ void load(const NsProduct& p, int z, int row, int col) {
        if constexpr (STAGE == kGram) return;
        in.load(p.in + (int64_t)z * p.stride_i, plane_index(row, p.ldi, col), p.plane_i);
    }
    // v: the accumulated sums on entry; on return the scaled values that are
    // stored (kGram, kPoly: for the mirrored store).  row_diag, col_diag: the
    // diagonal's entries of the row and the columns, where the stage reads
    // them (kPoly both, kUpdate the row's, kUpdateColumns the columns').
    __device__ __forceinline__ void finish(const NsProduct& p, int z, int row, int col, float row_diag,
                                           const float* col_diag, float (&v)[W]) const {
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] *= p.unscale;
        if constexpr (STAGE >= kUpdate) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float diag = STAGE == kUpdate ? row_diag : col_diag[e];
                v[e] = __builtin_fmaf(p.a + diag, in.value(e) * p.in_unscale, v[e]);
            }
            if (p.final_out != nullptr) {
                if (row < p.rows && col < p.cols)
                    store_values(p.final_type, p.final_out,
                                 (int64_t)z * p.final_stride + (int64_t)row * p.final_ld + col, p.cols - col, v);
                return;
            }
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] *= p.out_scale;
        } else {
            const int diag = row - col;                  // the run's entry on the diagonal, if any
            float on_diag = 0.0f;
            const bool has_diag = (unsigned)diag < (unsigned)W;
            if (has_diag) {
#pragma unroll
                for (int e = 0; e < W; ++e) on_diag = diag == e ? v[e] : on_diag;
            }
            if constexpr (STAGE == kPoly) {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const float s = in.value(e) * p.in_unscale;
                    v[e] = __builtin_fmaf(p.c, __builtin_fmaf(row_diag + col_diag[e], s, v[e]), p.b * s);
                }
            }
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] *= p.out_scale;
            if (has_diag) {
                if constexpr (STAGE == kPoly)
                    on_diag = __builtin_fmaf(p.c, __builtin_fmaf(row_diag, row_diag, on_diag), p.b * row_diag);
                p.diag_out[(int64_t)z * p.diag_n + row] = on_diag;
#pragma unroll
                for (int e = 0; e < W; ++e) v[e] = diag == e ? 0.0f : v[e];
            }
        }
        store_planes<W, LOW>(p.out + (int64_t)z * p.stride_o, plane_index(row, p.ldo, col), p.plane_o, v);
    }
};

// Tile t of a lower triangle of tiles, row by row.
__device__ __forceinline__ void triangle_tile(int t, int* tm, int* tn) {
    int m = (int)((__builtin_sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while ((m + 1) * (m + 2) / 2 <= t) ++m;
    while (m * (m + 1) / 2 > t) --m;
    *tm = m;
    *tn = t - m * (m + 1) / 2;
}

// The factors of matrix z.
__device__ __forceinline__ Gemm16Args ns_factors(const NsProduct& p, int z) {
    return Gemm16Args{p.M, p.N, p.K, p.A + (int64_t)z * p.stride_a, p.lda, p.B + (int64_t)z * p.stride_b, p.ldb,
                      nullptr, 0};
}

}  // namespace
#endif

}  // namespace gemmf32
