// newton_schulz_wide.hip -- the products of a Newton-Schulz step on the
// scheduled 256, 192 and 160 tiles (WideCore).
//
// X X^T and the square of a symmetric matrix are symmetric: only the tiles on
// and below the diagonal are computed, and a tile below it is stored twice,
// as it is and transposed.  The transposed store reads the finished values
// of 32 rows back from the patch column by column: four lanes on 32
// consecutive entries of a row of the result, 64 bytes per plane.
#include "epilogue.h"
#include "mfma16_wide_core.h"
#include "newton_schulz_product.h"
#include "staged_tile.h"

namespace gemmf32 {

namespace {

constexpr int kGroupM = 4;

template <bool KCA, bool KCB, int BT, int TERMS, int STAGE>
__global__ __launch_bounds__(256)
void ns_wide_kernel(NsProduct p, int tiles_m, int tiles_n, int tiles) {
    using Core = WideCore<1, KCA, KCB, BT, TERMS, true>;
    using Staged = StagedTile<Core::FM, Core::FN>;
    using Run = NsRun<STAGE, TERMS, 8>;
    constexpr bool SYMMETRIC = STAGE < kUpdate;
    // After the K loop: each wave's patch and slots, then the diagonal's
    // entries of the block's rows and columns.
    constexpr int NV = STAGE == kGram ? 0 : Run::LOW ? 2 : 1;
    constexpr int PATCHES = 4 * Staged::PATCH * 4, SLOTS = 4 * Staged::slot_bytes(NV);
    constexpr int EPILOGUE_BYTES = PATCHES + SLOTS + 2 * 4 * BT;
    constexpr int BYTES = EPILOGUE_BYTES > Core::LDS_BYTES ? EPILOGUE_BYTES : Core::LDS_BYTES;
    static_assert(BYTES <= 163840, "LDS");
    __shared__ __attribute__((aligned(16))) unsigned char lds[BYTES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int logical = xcd_contiguous((int)blockIdx.x, (int)gridDim.x);
    const int z = logical / tiles, t = logical - z * tiles;
    int tm, tn;
    if constexpr (SYMMETRIC) {
        triangle_tile(t, &tm, &tn);
    } else {
        const int group_size = kGroupM * tiles_n;
        const int g = t / group_size, first = g * kGroupM, gm = min(tiles_m - first, kGroupM), in_g = t - g * group_size;
        tm = first + in_g % gm;
        tn = in_g / gm;
    }
    const int m0 = tm * BT, n0 = tn * BT;
    floatx4 acc[Core::FM][Core::FN];
    Core::run(ns_factors(p, z), m0, n0, lds, acc, p.plane_a, p.plane_b);
    GEMM16_PIN_ACCUMULATORS(acc, Core::FM, Core::FN);
    __syncthreads();

    float* const patch = reinterpret_cast<float*>(lds) + wave * Staged::PATCH;
    u32x4* const slots = reinterpret_cast<u32x4*>(lds + PATCHES) + wave * (Staged::slot_bytes(NV) / 16);
    float* const row_diags = reinterpret_cast<float*>(lds + PATCHES + SLOTS);
    float* const col_diags = row_diags + BT;
    const int tid = threadIdx.x, wrow = wave / 2 * Core::WM, wcol = wave % 2 * Core::WN;
    const int row0 = m0 + wrow, col0 = n0 + wcol;
    if constexpr (STAGE != kGram) {
        const float* const d = p.diag_in + (int64_t)z * p.diag_n;
        if (tid < BT) {
            if constexpr (STAGE != kUpdateColumns) row_diags[tid] = m0 + tid < p.M ? d[m0 + tid] : 0.0f;
            if constexpr (STAGE != kUpdate) col_diags[tid] = n0 + tid < p.N ? d[n0 + tid] : 0.0f;
        }
        __syncthreads();
    }
    const bool mirror = SYMMETRIC && tm != tn;
    Staged::template rows<SYMMETRIC, NV>(
        acc, patch, slots, lane, true,
        [&](int row, int col, auto& pre) __attribute__((always_inline)) {
            if (row0 + row >= p.M || col0 + col >= p.N) return;
            Run run;
            run.load(p, z, row0 + row, col0 + col);
            if constexpr (NV > 0) __builtin_memcpy(&pre[0], run.in.h, 16);
            if constexpr (NV > 1) __builtin_memcpy(&pre[1], run.in.l, 16);
        },
        [&](int row, int col, float (&v)[8], const auto& pre) __attribute__((always_inline)) {
            if (row0 + row >= p.M || col0 + col >= p.N) return;
            Run run;
            if constexpr (NV > 0) __builtin_memcpy(run.in.h, &pre[0], 16);
            if constexpr (NV > 1) __builtin_memcpy(run.in.l, &pre[1], 16);
            run.finish(p, z, row0 + row, col0 + col, row_diags[wrow + row], col_diags + wcol + col, v);
        },
        [&](int first, int rows) __attribute__((always_inline)) {
            if (!mirror) return;
            const int q = 8 * (lane & 3);
#pragma unroll
            for (int k = 0; k < Core::WN / 16; ++k) {
                const int c = 16 * k + (lane >> 2);
                if (q >= rows || col0 + c >= p.N || row0 + first + q >= p.M) continue;
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = patch[(q + r) * Staged::PITCH + c];
                store_planes<8, Run::LOW>(p.out + (int64_t)z * p.stride_o,
                                          plane_index(col0 + c, p.ldo, row0 + first + q), p.plane_o, v);
            }
        });
}

template <int BT, int TERMS>
hipError_t launch(const NsProduct& p, int op_a, hipStream_t s) {
    const int tm = ceil_div(p.M, BT), tn = ceil_div(p.N, BT);
    const bool symmetric = p.stage < kUpdate;
    const int64_t tiles = symmetric ? (int64_t)tm * (tm + 1) / 2 : (int64_t)tm * tn;
    if (tiles * p.batch > 0x7FFFFFFFll / 256) return hipErrorInvalidValue;
    const dim3 g((unsigned)(tiles * p.batch)), b(256);
    const int t = (int)tiles;
    if (p.stage == kGram && op_a)
        hipLaunchKernelGGL((ns_wide_kernel<false, false, BT, TERMS, kGram>), g, b, 0, s, p, tm, tn, t);
    else if (p.stage == kGram) hipLaunchKernelGGL((ns_wide_kernel<true, true, BT, TERMS, kGram>), g, b, 0, s, p, tm, tn, t);
    else if (p.stage == kPoly) hipLaunchKernelGGL((ns_wide_kernel<true, true, BT, TERMS, kPoly>), g, b, 0, s, p, tm, tn, t);
    else if (p.stage == kUpdateColumns)
        hipLaunchKernelGGL((ns_wide_kernel<true, true, BT, TERMS, kUpdateColumns>), g, b, 0, s, p, tm, tn, t);
    else hipLaunchKernelGGL((ns_wide_kernel<true, false, BT, TERMS, kUpdate>), g, b, 0, s, p, tm, tn, t);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ns_wide(const NsProduct& p, int bt, int op_a, hipStream_t s) {
    if (p.terms == 1) {
        if (bt == 256) return launch<256, 1>(p, op_a, s);
        if (bt == 192) return launch<192, 1>(p, op_a, s);
        return launch<160, 1>(p, op_a, s);
    }
    if (bt == 256) return launch<256, 3>(p, op_a, s);
    if (bt == 192) return launch<192, 3>(p, op_a, s);
    return launch<160, 3>(p, op_a, s);
}

}  // namespace gemmf32
