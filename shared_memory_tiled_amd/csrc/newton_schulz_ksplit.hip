// newton_schulz_ksplit.hip -- the products of a Newton-Schulz step on 64 x 64
// tiles whose four waves split K (KsplitCore), for matrices whose large tiles
// would leave most compute units idle.  The symmetric products are computed
// whole: with one block per tile and fewer tiles than units, half of them
// would only idle.
//
// Built with the matrix instructions' vector-register form, as
// mfma16_ksplit.hip.
#include "epilogue.h"
#include "mfma16_ksplit_core.h"
#include "newton_schulz_product.h"

namespace gemmf32 {

namespace {

template <bool KCA, bool KCB, int TERMS, int STAGE>
__global__ __launch_bounds__(256)
void ns_ksplit_kernel(NsProduct p, int tiles_m, int tiles_n) {
    using Core = KsplitCore<1, KCA, KCB, TERMS>;
    __shared__ __attribute__((aligned(16))) uint16_t lds[Core::LDS_ELEMS];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int logical = xcd_contiguous((int)blockIdx.x, (int)gridDim.x);
    const int z = logical / (tiles_m * tiles_n), t = logical - z * (tiles_m * tiles_n);
    const int m0 = 64 * (t % tiles_m), n0 = 64 * (t / tiles_m);
    Core::run(ns_factors(p, z), m0, n0, lds, p.plane_a, p.plane_b);
    const int col = n0 + Core::sum_col(lane);
    const float* const d = STAGE == kGram ? nullptr : p.diag_in + (int64_t)z * p.diag_n;
    float col_diag[4], row_diag[4];
    if constexpr (STAGE == kPoly || STAGE == kUpdateColumns) __builtin_memcpy(col_diag, d + col, sizeof(col_diag));
    NsRun<STAGE, TERMS, 4> run[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int row = m0 + Core::sum_row(w, lane, it);
        if constexpr (STAGE == kPoly || STAGE == kUpdate) row_diag[it] = d[row];
        run[it].load(p, z, row, col);
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const floatx4 s = Core::sum4(lds, w, lane, it);
        float v[4] = {s[0], s[1], s[2], s[3]};
        run[it].finish(p, z, m0 + Core::sum_row(w, lane, it), col, row_diag[it], col_diag, v);
    }
}

template <int TERMS>
void launch(const NsProduct& p, int op_a, unsigned blocks, int tm, int tn, hipStream_t s) {
    const dim3 g(blocks), b(256);
    // S and T are symmetric: read mn-contiguous, in runs of 128 bytes instead
    // of 64.
    if (p.stage == kGram && op_a)
        hipLaunchKernelGGL((ns_ksplit_kernel<false, false, TERMS, kGram>), g, b, 0, s, p, tm, tn);
    else if (p.stage == kGram) hipLaunchKernelGGL((ns_ksplit_kernel<true, true, TERMS, kGram>), g, b, 0, s, p, tm, tn);
    else if (p.stage == kPoly) hipLaunchKernelGGL((ns_ksplit_kernel<false, false, TERMS, kPoly>), g, b, 0, s, p, tm, tn);
    else if (p.stage == kUpdateColumns)
        hipLaunchKernelGGL((ns_ksplit_kernel<true, false, TERMS, kUpdateColumns>), g, b, 0, s, p, tm, tn);
    else hipLaunchKernelGGL((ns_ksplit_kernel<false, false, TERMS, kUpdate>), g, b, 0, s, p, tm, tn);
}

}  // namespace

hipError_t launch_ns_ksplit(const NsProduct& p, int op_a, hipStream_t s) {
    const int tm = p.M / 64, tn = p.N / 64;
    const int64_t blocks = (int64_t)tm * tn * p.batch;
    if (blocks > 0x7FFFFFFFll / 256) return hipErrorInvalidValue;
    if (p.terms == 1) launch<1>(p, op_a, (unsigned)blocks, tm, tn, s);
    else launch<3>(p, op_a, (unsigned)blocks, tm, tn, s);
    return hipGetLastError();
}

}  // namespace gemmf32
