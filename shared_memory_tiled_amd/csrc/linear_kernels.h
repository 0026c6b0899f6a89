// linear_kernels.h -- launchers of the product kernels that end in an
// epilogue (epilogue.h), one family per translation unit (not part of the
// public interface).
#pragma once

#include "launch.h"

namespace gemmf32 {

// Each: op(A) op(B) into e (whose M and N end the result; p's may be one
// larger, for an even width of packed factors), format 0 bfloat16, 1 binary16, op 1: that factor
// stored transposed.  partials (gradient mode with column sums, else null):
// one row of e.N floats per tile row, written whole.
//   wide 256, 192, 160: what wide_fits takes, plus any K if both factors are
//   mn-contiguous (op_a 1, op_b 0)
//   ksplit, ksplit128: what ksplit16_fits and ksplit128_fits take, plus the same
hipError_t launch_linear_wide256(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                                 int op_b, float* partials);
hipError_t launch_linear_wide192(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                                 int op_b, float* partials);
hipError_t launch_linear_wide160(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                                 int op_b, float* partials);
hipError_t launch_linear_ksplit128(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                                   int op_b, float* partials);
hipError_t launch_linear_ksplit(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                                int op_b, float* partials);

// The 64 tiles with K split over blocks too: k_share (a multiple of 64) of K
// each, a plane of M x N floats per share.
hipError_t launch_linear_ksplit_planes(const Gemm16Args& p, int M, int N, hipStream_t s, int format, int op_a, int op_b,
                                       int k_share, float* planes);

// Few rows (linear_rows.hip): M <= kLinearRowsMax, A as stored, any alignment
// and sizes.  K is split over `splits` blocks; with one the epilogue runs in
// the kernel (forward mode), else the planes (M x N floats each) go to `planes`.
constexpr int kLinearRowsMax = 64;
int linear_rows_splits(int M, int N, int K);
hipError_t launch_linear_rows(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_b,
                              int splits, float* planes);
// Whether narrower blocks that take all of K and end in the epilogue (forward
// mode) are faster than K split over blocks, and their launcher.
bool linear_rows_fused(int M, int N, int K, int op_b);
hipError_t launch_linear_rows_fused(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_b);

}  // namespace gemmf32
