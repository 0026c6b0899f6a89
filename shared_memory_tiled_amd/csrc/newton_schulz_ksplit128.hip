// newton_schulz_ksplit128.hip -- the products of a Newton-Schulz step on
// 128 x 128 tiles whose four waves split K (Ksplit128Core), for matrices
// whose larger tiles fill the compute units badly.  Of the symmetric products
// the tiles on and below the diagonal are computed, as on the larger tiles
// (newton_schulz_wide.hip).
#include "epilogue.h"
#include "mfma16_ksplit128_core.h"
#include "mfma16_wide_core.h"
#include "newton_schulz_product.h"
#include "staged_tile.h"

namespace gemmf32 {

namespace {

template <bool KCA, bool KCB, int TERMS, int STAGE>
__global__ __launch_bounds__(256)
void ns_ksplit128_kernel(NsProduct p, int tiles_m, int tiles) {
    using Core = Ksplit128Core<1, KCA, KCB, TERMS>;
    using Run = NsRun<STAGE, TERMS, 4>;
    constexpr bool SYMMETRIC = STAGE < kUpdate;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Core::LDS_BYTES];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int logical = xcd_contiguous((int)blockIdx.x, (int)gridDim.x);
    const int z = logical / tiles, t = logical - z * tiles;
    int tm, tn;
    if constexpr (SYMMETRIC) {
        triangle_tile(t, &tm, &tn);
    } else {
        tm = t % tiles_m;
        tn = t / tiles_m;
    }
    const int m0 = 128 * tm, n0 = 128 * tn;
    floatx4 acc[8][8];
    Core::run(ns_factors(p, z), m0, n0, lds, acc, p.plane_a, p.plane_b);
    GEMM16_PIN_ACCUMULATORS(acc, 8, 8);
    // What the epilogue reads, a round ahead of its use.
    const int col = n0 + 4 * (lane & 31);
    const float* const d = STAGE == kGram ? nullptr : p.diag_in + (int64_t)z * p.diag_n;
    float col_diag[4], row_diag[8];
    if constexpr (STAGE == kPoly || STAGE == kUpdateColumns)
        if (col < p.N) __builtin_memcpy(col_diag, d + col, sizeof(col_diag));
    Run run[8];
    auto load = [&](int a, int it) __attribute__((always_inline)) {
        const int row = m0 + 16 * (4 * a + w) + 2 * it + (lane >> 5);
        if (row >= p.M || col >= p.N) return;
        if constexpr (STAGE == kPoly || STAGE == kUpdate) row_diag[it] = d[row];
        run[it].load(p, z, row, col);
    };
#pragma unroll
    for (int it = 0; it < 8; ++it) load(0, it);
    const bool mirror = SYMMETRIC && tm != tn;
    Core::exchange(
        acc, lds,
        [&](int a, int it, int r, int, floatx4 sum, float* slot) __attribute__((always_inline)) {
            float v[4] = {sum[0], sum[1], sum[2], sum[3]};
            if (m0 + r < p.M && col < p.N) run[it].finish(p, z, m0 + r, col, row_diag[it], col_diag, v);
            if (a == 0) load(1, it);
            if constexpr (SYMMETRIC) *reinterpret_cast<floatx4*>(slot) = floatx4{v[0], v[1], v[2], v[3]};
        },
        // The transposed store: two lanes on the 16 entries of a row of the
        // result that this wave's block row holds (row rho of it at float
        // 2048 w + 128 rho, columns XORed by 16 ((rho / 4) mod 2)).
        [&](int a) __attribute__((always_inline)) {
            if (!mirror) return;
            wave_lds_fence();
            const float* const rows = reinterpret_cast<const float*>(lds) + 2048 * w;
            const int q = 8 * (lane & 1), row0 = m0 + 16 * (4 * a + w) + q;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = 32 * k + (lane >> 1);
                if (n0 + c >= p.N || row0 >= p.M) continue;
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = rows[128 * (q + r) + (c ^ (16 * (((q + r) >> 2) & 1)))];
                store_planes<8, Run::LOW>(p.out + (int64_t)z * p.stride_o, plane_index(n0 + c, p.ldo, row0), p.plane_o, v);
            }
        });
}

template <int TERMS>
hipError_t launch(const NsProduct& p, int op_a, hipStream_t s) {
    const int tm = ceil_div(p.M, 128), tn = ceil_div(p.N, 128);
    const int64_t tiles = p.stage < kUpdate ? (int64_t)tm * (tm + 1) / 2 : (int64_t)tm * tn;
    if (tiles * p.batch > 0x7FFFFFFFll / 256) return hipErrorInvalidValue;
    const dim3 g((unsigned)(tiles * p.batch)), b(256);
    const int t = (int)tiles;
    // S and T are symmetric: read mn-contiguous, which these tiles copy in
    // runs of 256 bytes instead of 64 (2048^2, three terms, T: 74 us
    // k-contiguous, 60 so).
    if (p.stage == kGram && op_a)
        hipLaunchKernelGGL((ns_ksplit128_kernel<false, false, TERMS, kGram>), g, b, 0, s, p, tm, t);
    else if (p.stage == kGram) hipLaunchKernelGGL((ns_ksplit128_kernel<true, true, TERMS, kGram>), g, b, 0, s, p, tm, t);
    else if (p.stage == kPoly) hipLaunchKernelGGL((ns_ksplit128_kernel<false, false, TERMS, kPoly>), g, b, 0, s, p, tm, t);
    else if (p.stage == kUpdateColumns)
        hipLaunchKernelGGL((ns_ksplit128_kernel<true, false, TERMS, kUpdateColumns>), g, b, 0, s, p, tm, t);
    else hipLaunchKernelGGL((ns_ksplit128_kernel<false, false, TERMS, kUpdate>), g, b, 0, s, p, tm, t);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_ksplit128(const NsProduct& p, int op_a, hipStream_t s) {
    return p.terms == 1 ? launch<1>(p, op_a, s) : launch<3>(p, op_a, s);
}

}  // namespace gemmf32
