// staged_tile.h -- a wave's accumulators of 16 x 16 blocks handed on as runs
// of consecutive columns, through LDS (device code shared by the kernels on
// WideCore that end in an epilogue; not part of the public interface).
//
// An accumulator register holds one column of four rows per lane group; a
// 16-bit store of it would touch 32 bytes of a row.  Two block rows (32 rows)
// of a wave at a time go through a patch of LDS of its own, written as
// accumulated (row pitch 4 floats over the width: the four lane groups' rows
// lie 16 banks apart, conflict free) and read back as 8 consecutive columns
// per lane, so that every global access of the epilogue is 16 bytes or more
// and a row of a 256 tile's wave is one run of 256 bytes of 16-bit values.
//
// What the epilogue reads from memory (a residual, a pre-activation, the
// other term of a sum) comes a group ahead: loaded into registers while the
// group before is worked on, then put into the lane's own slots of LDS, so
// that the loop over a group's runs can stay rolled.  With one wave per SIMD
// nothing else hides the latency, and the counter that a load is waited for
// with counts the stores too: a load in the loop makes each run wait for the
// stores before it (20 us of a 256 x 256 tile's epilogue; so do loads that are
// never reached, which is why edges have a loop of their own).  One vector per
// run is loaded for the whole tile before the first store, two a group at a
// time.
#pragma once

#include "mfma16_common.h"

namespace gemmf32 {

namespace {

// Orders a wave's LDS accesses: what its lanes wrote before is visible to
// all of them after (LDS serves a wave's accesses in order).
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float read_accumulator(float a) {
    float v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
}

template <int FM, int FN>
struct StagedTile {
    static constexpr int W = 16 * FN, PITCH = W + 4;
    static constexpr int PATCH = 32 * PITCH;              // floats per wave
    static constexpr int CHUNKS = W / 8;                  // runs of 8 columns per row
    static constexpr int GROUPS = (FM + 1) / 2;           // of 32 rows (the last of 16 if FM is odd)
    static constexpr int ITERS = CHUNKS / 2;              // runs of a lane in a full group
    static constexpr int LAST_ITERS = FM % 2 ? (CHUNKS + 3) / 4 : ITERS;
    static constexpr int RUNS = (GROUPS - 1) * ITERS + LAST_ITERS;
    static_assert(CHUNKS % 2 == 0, "whole runs in a full group");

    // Run t of a lane: its number within the group, row and column in the
    // wave's span; false past the last row.
    __device__ static __forceinline__ bool run_at(int t, int lane, int* it, int* row, int* col) {
        const int g = t / ITERS;
        *it = t - g * ITERS;
        const int id = 64 * *it + lane;
        const int r = id / CHUNKS;
        *row = 32 * g + r;
        *col = 8 * (id - r * CHUNKS);
        return *row < 16 * FM;
    }

    // Bytes of a wave's slots for NV vectors of 16 bytes per run.
    static constexpr int slot_bytes(int nv) { return ITERS * 64 * 16 * nv; }

    // For every run: use(row, col, v, pre) with v[8] the columns col .. col +
    // 7 and pre[NV] what load(row, col, pre) brought (only if `loads`, the
    // same for every lane); what use leaves in v is written back to the patch
    // if WRITE_BACK, and done(row0, rows) runs after the `rows` rows of a group
    // from row0 (patch row 0).  Both see runs inside the wave's span only.
    template <bool WRITE_BACK, int NV, typename L, typename F, typename G>
    __device__ static __forceinline__ void rows(const floatx4 (&acc)[FM][FN], float* patch, u32x4* slots, int lane,
                                                bool loads, L&& load, F&& use, G&& done) {
        float* const wr = patch + 4 * (lane >> 4) * PITCH + (lane & 15);
        constexpr int V = NV > 0 ? NV : 1;
        constexpr int HELD = NV == 1 ? RUNS : ITERS;          // runs held in registers
        u32x4 ahead[HELD][V];
        auto fetch = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                int it, row, col;
                if (t0 + i < RUNS && run_at(t0 + i, lane, &it, &row, &col)) load(row, col, ahead[i]);
            }
        };
        if (NV > 0 && loads) fetch(0);
        unroll<GROUPS>([&](auto gc) __attribute__((always_inline)) {
            constexpr int g = decltype(gc)::value;
            if (NV > 0 && loads) {
#pragma unroll
                for (int i = 0; i < ITERS; ++i)
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (g * ITERS + i < RUNS) slots[(i * V + k) * 64 + lane] = ahead[NV == 1 ? g * ITERS + i : i][k];
                if (NV != 1 && g + 1 < GROUPS) fetch((g + 1) * ITERS);
            }
            wave_lds_fence();
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (2 * g + b < FM) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int j = 0; j < FN; ++j)
                            wr[(16 * b + r) * PITCH + 16 * j] = acc[2 * g + b < FM ? 2 * g + b : 0][j][r];
                }
            wave_lds_fence();
#pragma unroll 1
            for (int i = 0; i < (g == GROUPS - 1 ? LAST_ITERS : ITERS); ++i) {
                int it, row, col;
                if (run_at(g * ITERS + i, lane, &it, &row, &col)) {
                    u32x4 pre[V];
                    if (NV > 0 && loads) {
#pragma unroll
                        for (int k = 0; k < V; ++k) pre[k] = slots[(i * V + k) * 64 + lane];
                    }
                    floatx4* q = reinterpret_cast<floatx4*>(patch + (row - 32 * g) * PITCH + col);
                    const floatx4 lo = q[0], hi = q[1];
                    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    use(row, col, v, pre);
                    if constexpr (WRITE_BACK) {
                        q[0] = floatx4{v[0], v[1], v[2], v[3]};
                        q[1] = floatx4{v[4], v[5], v[6], v[7]};
                    }
                }
            }
            if constexpr (WRITE_BACK) wave_lds_fence();
            done(32 * g, 2 * g + 1 < FM ? 32 : 16);
        });
    }
};

}  // namespace

}  // namespace gemmf32
