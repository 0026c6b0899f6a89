// grouped_tiles.h -- the tiles of the grouped layer on the library's scheduled
// K loops (WideCore, Ksplit128Core, KsplitCore), instantiated per tile size in
// grouped_wide*.hip and grouped_ksplit*.hip (device code; not part of the
// public interface).
//
// A block finds its group, enters the group's rows and weight as a product of
// their own and runs the K loop of the plain product on it; the epilogue is the
// layer's forward one.  The group's rows begin at the tile's first row, so only
// a tile's extent has to fit the copies' 32-bit offsets.
#pragma once

#include "epilogue.h"
#include "grouped_kernels.h"
#include "mfma16_wide_core.h"
#include "staged_tile.h"

namespace gemmf32 {

namespace {

// Zeros over the block's BT x BT tile at (m0, n0): the gradient of a weight
// that no row chose.
template <int BT>
__device__ __forceinline__ void zero_tile(const EpilogueArgs& e, int m0, int n0) {
    const float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = threadIdx.x; i < BT * BT / 8; i += 256) {
        const int row = m0 + i / (BT / 8), col = n0 + 8 * (i % (BT / 8));
        if (row < e.M && col < e.N) store_values(e.c_type, e.C, (int64_t)row * e.ldc + col, e.N - col, v);
    }
}

// The forward epilogue on WideCore's accumulators, from behind the barrier that
// ends the K loop: through LDS as runs of 8 columns (StagedTile); thread t holds
// bias value n0 + t.  Whole runs with places of 32 bits and a 16-bit residual
// loaded for the whole tile ahead of the first store; else (N no multiple of 8
// at the edge, a binary32 residual) a loop that loads where it uses.
template <typename Core>
struct WideForward {
    using Staged = StagedTile<Core::FM, Core::FN>;
    using Run = EpilogueRun<8, false>;
    static constexpr int BT = Core::BM;
    static constexpr int PATCHES = 4 * Staged::PATCH * 4, SLOTS = 4 * Staged::slot_bytes(1);
    static constexpr int BYTES =
        PATCHES + SLOTS + 4 * BT > Core::LDS_BYTES ? PATCHES + SLOTS + 4 * BT : Core::LDS_BYTES;
    static_assert(BYTES <= 163840, "LDS");

    __device__ static __forceinline__ void finish(const floatx4 (&acc)[Core::FM][Core::FN], const EpilogueArgs& e,
                                                  int m0, int n0, float bias, unsigned char* lds) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        float* const shared = reinterpret_cast<float*>(lds + PATCHES + SLOTS);
        if ((int)threadIdx.x < BT) shared[threadIdx.x] = bias;
        __syncthreads();
        float* const patch = reinterpret_cast<float*>(lds) + wave * Staged::PATCH;
        const int row0 = m0 + wave / 2 * Core::WM, wcol = wave % 2 * Core::WN, col0 = n0 + wcol;
        u32x4* const slots = reinterpret_cast<u32x4*>(lds + PATCHES) + wave * (Staged::slot_bytes(1) / 16);
        const bool residual = e.residual != nullptr;
        auto bias_of = [&](int col, float (&b)[8]) __attribute__((always_inline)) {
            const floatx4 lo = *reinterpret_cast<const floatx4*>(shared + wcol + col);
            const floatx4 hi = *reinterpret_cast<const floatx4*>(shared + wcol + col + 4);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                b[c] = lo[c];
                b[4 + c] = hi[c];
            }
        };
        constexpr int64_t kMaxLd = 1 << 22;
        if ((n0 + BT <= e.N || e.N % 8 == 0) && !(residual && e.c_type == 2) && e.ldc < kMaxLd &&
            (!residual || e.ldr < kMaxLd) && (e.preact == nullptr || e.ldz < kMaxLd)) {
            char* const c_base = static_cast<char*>(e.C) + (e.c_type == 2 ? 4 : 2) * ((int64_t)row0 * e.ldc + col0);
            char* const z_base = static_cast<char*>(e.preact) + 2 * ((int64_t)row0 * e.ldz + col0);
            const char* const r_base = static_cast<const char*>(e.residual) + 2 * ((int64_t)row0 * e.ldr + col0);
            const unsigned ldc = (unsigned)e.ldc, ldz = (unsigned)e.ldz, ldr = (unsigned)e.ldr;
            Staged::template rows<false, 1>(
                acc, patch, slots, lane, residual,
                [&](int row, int col, u32x4 (&pre)[1]) __attribute__((always_inline)) {
                    if (row0 + row >= e.M || col0 + col >= e.N) return;
                    __builtin_memcpy(&pre[0], r_base + 2 * (__umul24(row, ldr) + col), 16);
                },
                [&](int row, int col, float (&v)[8], const u32x4 (&pre)[1]) __attribute__((always_inline)) {
                    if (row0 + row >= e.M || col0 + col >= e.N) return;
                    float b[8];
                    bias_of(col, b);
                    Run run;
                    __builtin_memcpy(run.residual.w, &pre[0], 16);
                    run.finish_at(e, c_base, __umul24(row, ldc) + col, z_base, __umul24(row, ldz) + col, b, v);
                },
                [](int, int) {});
        } else {
            Staged::template rows<false, 0>(
                acc, patch, slots, lane, false, [](int, int, u32x4 (&)[1]) {},
                [&](int row, int col, float (&v)[8], const u32x4 (&)[1]) __attribute__((always_inline)) {
                    if (row0 + row >= e.M || col0 + col >= e.N) return;
                    float b[8];
                    bias_of(col, b);
                    Run run;
                    run.load(e, row0 + row, col0 + col);
                    run.finish(e, row0 + row, col0 + col, b, v);
                },
                [](int, int) {});
        }
    }
};

template <int FMT, bool KCB, int BT>
__global__ __launch_bounds__(256)
void grouped_wide_kernel(GroupedArgs a, Gemm16Args p, EpilogueArgs e, int tiles_n, int group_m) {
    using Core = WideCore<FMT, true, KCB, BT>;
    using Forward = WideForward<Core>;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Forward::BYTES];
    const GroupRows r = locate_group_tile<BT>(a, (int)blockIdx.x, tiles_n, group_m);
    if (r.rows < 0) return;
    enter_group(a, r, &p, &e);
    const int m0 = BT * r.tm, n0 = BT * r.tn;
    p.A += (int64_t)m0 * p.lda;
    p.M = min(r.rows - m0, BT);
    float bias[1] = {0.0f};
    if ((int)threadIdx.x < BT) load_bias(e, n0 + (int)threadIdx.x, bias);
    floatx4 acc[Core::FM][Core::FN];
    Core::run(p, 0, n0, lds, acc);
    GEMM16_PIN_ACCUMULATORS(acc, Core::FM, Core::FN);
    __syncthreads();
    Forward::finish(acc, e, m0, n0, bias[0], lds);
}

// The weights' gradient: block -> (group, tile), the tiles of a group shared by
// the XCDs (groups differ in their rows; whole groups to an XCD would not
// balance).
template <int FMT, int BT>
__global__ __launch_bounds__(256)
void grouped_grad_wide_kernel(GroupedArgs a, Gemm16Args p, EpilogueArgs e, int tiles_m, int tiles_n, int group_m) {
    using Core = WideCore<FMT, false, false, BT>;
    using Forward = WideForward<Core>;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Forward::BYTES];
    const GroupRows r = locate_grad_tile(a, (int)blockIdx.x, tiles_m, tiles_n, group_m);
    enter_grad_group(a, r, &p, &e);
    const int m0 = BT * r.tm, n0 = BT * r.tn;
    if (r.rows == 0) return zero_tile<BT>(e, m0, n0);
    floatx4 acc[Core::FM][Core::FN];
    Core::run(p, m0, n0, lds, acc);
    GEMM16_PIN_ACCUMULATORS(acc, Core::FM, Core::FN);
    __syncthreads();
    Forward::finish(acc, e, m0, n0, 0.0f, lds);
}

template <int BT>
hipError_t launch_wide(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format,
                       int op_b) {
    constexpr int kGroupM = 4;                                     // as the plain product's launches
    const int tn = ceil_div(p.N, BT);
    const dim3 g((unsigned)(grouped_row_tiles(a.rows, a.groups, BT) * tn)), b(256);
    if (format == 0 && op_b) hipLaunchKernelGGL((grouped_wide_kernel<0, true, BT>), g, b, 0, s, a, p, e, tn, kGroupM);
    else if (format == 0) hipLaunchKernelGGL((grouped_wide_kernel<0, false, BT>), g, b, 0, s, a, p, e, tn, kGroupM);
    else if (op_b) hipLaunchKernelGGL((grouped_wide_kernel<1, true, BT>), g, b, 0, s, a, p, e, tn, kGroupM);
    else hipLaunchKernelGGL((grouped_wide_kernel<1, false, BT>), g, b, 0, s, a, p, e, tn, kGroupM);
    return hipGetLastError();
}

template <int BT>
hipError_t launch_grad_wide(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format) {
    constexpr int kGroupM = 4;
    const int tm = ceil_div(p.M, BT), tn = ceil_div(p.N, BT);
    const dim3 g((unsigned)(tm * tn * a.groups)), b(256);
    if (format == 0) hipLaunchKernelGGL((grouped_grad_wide_kernel<0, BT>), g, b, 0, s, a, p, e, tm, tn, kGroupM);
    else hipLaunchKernelGGL((grouped_grad_wide_kernel<1, BT>), g, b, 0, s, a, p, e, tm, tn, kGroupM);
    return hipGetLastError();
}

}  // namespace

}  // namespace gemmf32
