// linear_wide_kernel.h -- the product with its epilogue on the scheduled 256,
// 192 and 160 tiles (WideCore), instantiated per tile size in
// linear_wide*.hip (device code; not part of the public interface).
//
// The K loop is mfma16_wide.hip's; then the accumulators go through LDS as
// runs of 8 consecutive columns (staged_tile.h), the bias from LDS, residual
// and pre-activation from memory a group of rows ahead, so that a 16-bit
// result is written in rows of 256 bytes and nothing passes through memory in
// binary32.  Tiles across column N with N no multiple of 8, and binary32
// residuals, take a second loop that loads where it uses.
// The column sums of the gradient mode are taken column by column from what
// each group of 32 rows leaves in LDS, then added over the block's two row
// halves, in a fixed order.
#pragma once

#include "epilogue.h"
#include "linear_kernels.h"
#include "mfma16_wide_core.h"
#include "staged_tile.h"

namespace gemmf32 {

namespace {

template <int FMT, bool KCA, bool KCB, int BT, bool GRADIENT>
__global__ __launch_bounds__(256)
void linear_wide_kernel(Gemm16Args p, EpilogueArgs e, int tiles_m, int tiles_n, int group_m, float* partials) {
    using Core = WideCore<FMT, KCA, KCB, BT>;
    using Staged = StagedTile<Core::FM, Core::FN>;
    using Run = EpilogueRun<8, GRADIENT>;
    // After the K loop: each wave's patch and slots, then BT floats.  Slots: a
    // 16-bit residual and, in gradient mode, the pre-activation.
    constexpr int NV = GRADIENT ? 2 : 1;
    constexpr int PATCHES = 4 * Staged::PATCH * 4, SLOTS = 4 * Staged::slot_bytes(NV);
    constexpr int BYTES = PATCHES + SLOTS + 4 * BT > Core::LDS_BYTES ? PATCHES + SLOTS + 4 * BT : Core::LDS_BYTES;
    static_assert(BYTES <= 163840, "LDS");
    __shared__ __attribute__((aligned(16))) unsigned char lds[BYTES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int tm, tn;
    grouped_tile((int)blockIdx.x, tiles_m, tiles_n, group_m, &tm, &tn);
    const int m0 = tm * BT, n0 = tn * BT;
    float bias[1] = {0.0f};
    if constexpr (!GRADIENT)
        if ((int)threadIdx.x < BT) load_bias(e, n0 + (int)threadIdx.x, bias);
    floatx4 acc[Core::FM][Core::FN];
    Core::run(p, m0, n0, lds, acc);
    GEMM16_PIN_ACCUMULATORS(acc, Core::FM, Core::FN);
    __syncthreads();

    float* const shared = reinterpret_cast<float*>(lds + PATCHES + SLOTS);
    if constexpr (!GRADIENT) {
        if ((int)threadIdx.x < BT) shared[threadIdx.x] = bias[0];
        __syncthreads();
    }
    float* const patch = reinterpret_cast<float*>(lds) + wave * Staged::PATCH;
    const int row0 = m0 + wave / 2 * Core::WM, wcol = wave % 2 * Core::WN, col0 = n0 + wcol;
    float sums[2] = {0.0f, 0.0f};                  // of columns lane, lane + 64 of the wave's
    u32x4* const slots = reinterpret_cast<u32x4*>(lds + PATCHES) + wave * (Staged::slot_bytes(NV) / 16);
    const bool residual = e.residual != nullptr, z = GRADIENT && e.act != kActNone;
    auto bias_of = [&](int col, float (&b)[8]) __attribute__((always_inline)) {
        if constexpr (!GRADIENT) {
            const floatx4 lo = *reinterpret_cast<const floatx4*>(shared + wcol + col);
            const floatx4 hi = *reinterpret_cast<const floatx4*>(shared + wcol + col + 4);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                b[c] = lo[c];
                b[4 + c] = hi[c];
            }
        }
    };
    auto outside = [&](int row, int col, float (&v)[8]) __attribute__((always_inline)) -> bool {
        if (row0 + row < e.M && col0 + col < e.N) return false;
        if constexpr (GRADIENT) {
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = 0.0f;                // for the column sums
        }
        return true;
    };
    auto column_sums = [&](int, int rows) __attribute__((always_inline)) {
        if constexpr (GRADIENT) {
            if (partials == nullptr) return;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = lane + 64 * h;
                if (c < Core::WN) {
#pragma unroll 8
                    for (int r = 0; r < rows; ++r) sums[h] += patch[r * Staged::PITCH + c];
                }
            }
        }
    };
    // Places within a wave's span as 32-bit offsets from its corner.
    constexpr int64_t kMaxLd = 1 << 22;
    if ((n0 + BT <= e.N || e.N % 8 == 0) && !(residual && e.c_type == 2) && e.ldc < kMaxLd &&
        (!residual || e.ldr < kMaxLd) && (e.preact == nullptr || e.ldz < kMaxLd)) {
        char* const c_base = static_cast<char*>(e.C) + (e.c_type == 2 ? 4 : 2) * ((int64_t)row0 * e.ldc + col0);
        char* const z_base = static_cast<char*>(e.preact) + 2 * ((int64_t)row0 * e.ldz + col0);
        const char* const r_base = static_cast<const char*>(e.residual) + 2 * ((int64_t)row0 * e.ldr + col0);
        const unsigned ldc = (unsigned)e.ldc, ldz = (unsigned)e.ldz, ldr = (unsigned)e.ldr;
        Staged::template rows<GRADIENT, NV>(
            acc, patch, slots, lane, residual || z,
            [&](int row, int col, u32x4 (&pre)[NV]) __attribute__((always_inline)) {
                if (row0 + row >= e.M || col0 + col >= e.N) return;
                if (residual) __builtin_memcpy(&pre[0], r_base + 2 * (__umul24(row, ldr) + col), 16);
                if (z) __builtin_memcpy(&pre[NV - 1], z_base + 2 * (__umul24(row, ldz) + col), 16);
            },
            [&](int row, int col, float (&v)[8], const u32x4 (&pre)[NV]) __attribute__((always_inline)) {
                if (outside(row, col, v)) return;
                float b[8];
                bias_of(col, b);
                Run run;
                __builtin_memcpy(run.residual.w, &pre[0], 16);
                if constexpr (GRADIENT) __builtin_memcpy(run.preact, &pre[NV - 1], 16);
                run.finish_at(e, c_base, __umul24(row, ldc) + col, z_base, __umul24(row, ldz) + col, b, v);
            },
            column_sums);
    } else {
        Staged::template rows<GRADIENT, 0>(
            acc, patch, slots, lane, false, [](int, int, u32x4 (&)[1]) {},
            [&](int row, int col, float (&v)[8], const u32x4 (&)[1]) __attribute__((always_inline)) {
                if (outside(row, col, v)) return;
                float b[8];
                bias_of(col, b);
                Run run;
                run.load(e, row0 + row, col0 + col);
                run.finish(e, row0 + row, col0 + col, b, v);
            },
            column_sums);
    }
    if constexpr (GRADIENT) {
        if (partials == nullptr) return;                            // the same for every thread
        if (wave >= 2) {                                            // the lower rows' half
            shared[wcol + lane] = sums[0];
            if (lane + 64 < Core::WN) shared[wcol + lane + 64] = sums[1];
        }
        __syncthreads();
        if (wave < 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = lane + 64 * h;
                if (c < Core::WN && col0 + c < e.N)
                    partials[(int64_t)tm * e.N + col0 + c] = sums[h] + shared[wcol + c];
            }
        }
    }
}

template <int FMT, bool KCA, bool KCB, int BT>
void launch_linear_wide_ops(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int tm, int tn, int group_m,
                            float* partials) {
    const dim3 g((unsigned)(tm * tn)), b(256);
    if (e.gradient)
        hipLaunchKernelGGL((linear_wide_kernel<FMT, KCA, KCB, BT, true>), g, b, 0, s, p, e, tm, tn, group_m, partials);
    else
        hipLaunchKernelGGL((linear_wide_kernel<FMT, KCA, KCB, BT, false>), g, b, 0, s, p, e, tm, tn, group_m, partials);
}

template <int BT>
hipError_t launch_linear_wide(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a, int op_b,
                              float* partials) {
    constexpr int kGroupM = 4;                                     // as mfma16_wide.hip's launches
    const int tm = ceil_div(p.M, BT), tn = ceil_div(p.N, BT);
    if ((int64_t)tm * tn > 0x7FFFFFFFll / 256) return hipErrorInvalidValue;
    switch (4 * (format ? 1 : 0) + 2 * (op_a ? 1 : 0) + (op_b ? 1 : 0)) {
        case 0: launch_linear_wide_ops<0, true, false, BT>(p, e, s, tm, tn, kGroupM, partials); break;
        case 1: launch_linear_wide_ops<0, true, true, BT>(p, e, s, tm, tn, kGroupM, partials); break;
        case 2: launch_linear_wide_ops<0, false, false, BT>(p, e, s, tm, tn, kGroupM, partials); break;
        case 3: launch_linear_wide_ops<0, false, true, BT>(p, e, s, tm, tn, kGroupM, partials); break;
        case 4: launch_linear_wide_ops<1, true, false, BT>(p, e, s, tm, tn, kGroupM, partials); break;
        case 5: launch_linear_wide_ops<1, true, true, BT>(p, e, s, tm, tn, kGroupM, partials); break;
        case 6: launch_linear_wide_ops<1, false, false, BT>(p, e, s, tm, tn, kGroupM, partials); break;
        default: launch_linear_wide_ops<1, false, true, BT>(p, e, s, tm, tn, kGroupM, partials); break;
    }
    return hipGetLastError();
}

}  // namespace

}  // namespace gemmf32
