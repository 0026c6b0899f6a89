// linear_w4.hip -- the product of a few rows with a weight held in 4 bits
// (a decoder's tokens), with the layer's epilogue.
//
//   Z[i][n] = sum over groups j of s[n][j] sum over k in j of
//             x[i][k] (q[n][k] - z[n][j]),     C = act(Z + bias) + residual
//
// The weight's bytes set the time, so it goes from memory straight into
// registers, and into matrix operands with one operation per value: q in the
// upper bits of a 16-bit float's fraction reads as 16 + q, exactly, and the 16
// is taken out together with the zero point,
//   sum x (q - z) = sum x (16 + q) - (16 + z) sum x,
// where sum x comes from one more matrix product, with ones, per 32 k: it lands
// in the registers where the rows' sums are.  The scale multiplies the group's
// binary32 sum: no weight is rounded.  The sums are rounded relative to |x| (16 + q)
// and |x| (16 + z), together 12 times |x (q - 8)| for q spread evenly and 24 for
// normal weights with the largest of 128 at 7: measured against binary64 (16 x
// 512 x 4096, 128 k to a scale, f32 out, root mean square of the result) 1.1e-7 and
// 2.0e-7 in bf16, 2.4e-7 and 4.6e-7 in f16, where products of the same whole
// numbers in 16 bits leave 6e-8 and 8e-8.  A 16-bit result's own rounding is 450
// times as much and more.  Range: below |x| = 2^116 no sum of 128 passes 2^128.
//
// A step is 128 k.  Lane (c = l % 16, g = l / 16) loads 16 bytes, 32 values,
// of column c from k 32 g on; a 4 x 4 transpose of dwords across the four lane
// groups (four lane swaps) then gives it, for each slice of 32 k, the eight
// values from 8 g on, as v_mfma_f32_16x16x32 takes them -- so that a matrix
// instruction stays inside one slice and so inside one scale group.  The pairs
// that a mask cuts out of a dword are values e and e + 4; x's eight values are
// put in that order (0 4 1 5 2 6 3 7).
//
// Up to 16 rows (linear_w4_kernel) the waves of a block split K, each a run of
// whole steps, and add their sums in LDS in wave order.  More rows
// (linear_w4_tile_kernel) would have every wave read all of x, many times the
// weight's bytes: there a block's four waves take 32 columns each of the same k
// and share x's step through LDS.  In both, few columns split K over blocks too:
// each stores its plane of sums and the epilogue pass adds them in order.
// Columns past N and rows past M repeat the last one and are not stored; values
// of x past K are zero, whatever the weight's bytes hold there.
//
// Measured in a graph, 128 k to a scale: 1 x 4096 x 4096 bf16 6.9 us (7.3 with the
// weight in memory; a launch, one load's latency and a block's sum), 1 x 8192 x
// 8192 11.6 (15.3, 2.3 TB/s), 16 x 8192 x 8192 16.5, 64 x 4096 x 4096 13.4, 256 x
// 4096 x 4096 26 to 29.  The expansion does not bound it (without it 16 x 8192 x 8192
// f16 with 64 k to a scale 17.5 for 17.7, 256 x 4096 x 4096 27 for 26): up to 16 rows
// each wave reads 4 KB of x per step for 2 KB of weight (without x 12.0) and, one to
// a SIMD, waits for its steps' loads; more rows take a barrier a step.
#include "epilogue.h"
#include "linear_w4.h"
#include "mfma16_common.h"

namespace gemmf32 {

namespace {

constexpr int kStep = 128;

template <int FMT>
struct W4 {
    // 16 + q: the exponent of 16 and q below it
    static constexpr unsigned BASE = FMT == 0 ? 0x41804180u : 0x4C004C00u;
    static constexpr unsigned ONES = FMT == 0 ? 0x3F803F80u : 0x3C003C00u;
    static constexpr int SHIFT = FMT == 0 ? 3 : 6;        // q's place in the fraction
    static constexpr unsigned MASK = 0x000F000Fu << SHIFT;
    // The mask and BASE come in registers: v_and_or_b32 takes no literals.
    __device__ static __forceinline__ u32x4 expand(unsigned w, unsigned mask, unsigned base) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {                      // values i and i + 4
            const unsigned v = SHIFT >= 4 * i ? w << (SHIFT >= 4 * i ? SHIFT - 4 * i : 0)
                                              : w >> (SHIFT >= 4 * i ? 0 : 4 * i - SHIFT);
            r[i] = (v & mask) | base;
        }
        return r;
    }
    // Eight values in the order 0 4 1 5 2 6 3 7.
    __device__ static __forceinline__ u32x4 reorder(u32x4 x) {
        return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                     __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
    }
    __device__ static __forceinline__ float value(unsigned bits) {
        if constexpr (FMT == 0) return __builtin_bit_cast(float, bits << 16);
        else return (float)__builtin_bit_cast(_Float16, (unsigned short)bits);
    }
};

// v[i] of lane group g <-> v[g] of lane group i (groups of 16 lanes).
__device__ __forceinline__ void transpose_groups(u32x4& v) {
    auto swap32 = [](unsigned a, unsigned b) { return __builtin_amdgcn_permlane32_swap(a, b, false, false); };
    auto swap16 = [](unsigned a, unsigned b) { return __builtin_amdgcn_permlane16_swap(a, b, false, false); };
    const auto p = swap32(v[0], v[2]), q = swap32(v[1], v[3]);
    const auto r = swap16(p[0], q[0]), s = swap16(p[1], q[1]);
    v = u32x4{r[0], r[1], s[0], s[1]};
}

// Eight consecutive 16-bit values from k on of a row of `count`, zeros past its
// end: one load of 16 bytes that stays inside the row, moved down to its place.
__device__ __forceinline__ u32x4 load_edge(const uint16_t* row, int k, int count) {
    u32x4 v = {0, 0, 0, 0};
    if (count < 8) {                                       // the same for every lane
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const unsigned u = row[min(k + e, count - 1)];
            v[e / 2] |= (k + e < count ? u : 0u) << (16 * (e % 2));
        }
        return v;
    }
    const int from = min(k, count - 8);
    __builtin_memcpy(&v, row + from, 16);
    return move_down(v, k - from);
}

// The scales or zero points of COLS columns for GROUPS groups, in LDS: read from
// memory by rows, since a wave's 16 columns touch 16 cache lines whatever little
// they read (one load of 2 bytes per step, column tile and kind took a third of
// 16 x 8192 x 8192's time: 24 us with them, 16 without).  Rows are padded so that
// 16 columns' values lie on different banks.
template <int COLS, int GROUPS>
struct GroupValues {
    static constexpr int PITCH = GROUPS + 4;
    uint16_t v[COLS][PITCH];
    // `count` groups from `first` on of the columns from n0 on, of rows of `total`.
    __device__ __forceinline__ void fill(const uint16_t* base, int64_t ld, int n0, int N, int first, int count, int total) {
        const int runs = (count + 7) / 8, shift = runs > 1 ? 32 - __builtin_clz(runs - 1) : 0;
        for (int i = threadIdx.x; i < COLS << shift; i += blockDim.x) {
            const int c = i >> shift, at = 8 * (i & ((1 << shift) - 1));
            if (at >= 8 * runs) continue;
            const u32x4 r = load_edge(base + (int64_t)min(n0 + c, N - 1) * ld, first + at, total);
            u32x2* const to = reinterpret_cast<u32x2*>(&v[c][at]);
            to[0] = u32x2{r[0], r[1]};
            to[1] = u32x2{r[2], r[3]};
        }
    }
};

// What a wave reads of its J tiles of 16 columns from memory for a step: the
// weight's bytes.
template <int J>
struct Weights {
    u32x4 q[J];
};
// SLICES: slices of 32 k per scale within a step (1, 2, or 4 for groups of 128 and
// more), so 4 / SLICES scales.
template <int J, int SLICES>
struct Columns {
    const uint8_t* q[J];
    int g, group_steps;
    // Columns from n0 on; those past N repeat the last one.
    __device__ __forceinline__ Columns(const W4Args& p, int n0, int lane) : g(lane >> 4), group_steps(p.group / kStep) {
#pragma unroll
        for (int j = 0; j < J; ++j) q[j] = p.Q + (int64_t)min(n0 + 16 * j + (lane & 15), p.N - 1) * p.ldq + 16 * g;
    }
    __device__ __forceinline__ int group_of(int step) const {
        if constexpr (SLICES < 4) return step * (4 / SLICES);
        return group_steps == 1 ? step : (int)((unsigned)step / (unsigned)group_steps);
    }
    // A step that lies inside K.
    __device__ __forceinline__ void load(Weights<J>& w, int step) const {
#pragma unroll
        for (int j = 0; j < J; ++j) __builtin_memcpy(&w.q[j], q[j] + step * (kStep / 2), 16);
    }
    // The step across K: what lies past it meets zeros of x, so only reads past a
    // row's end matter.  Four bytes at a time, inside the row and moved down.
    __device__ __forceinline__ void load_last(Weights<J>& w, int K, int step) const {
        const int at = step * (kStep / 2) + 16 * g, bytes = K / 2 + K % 2;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint8_t* const row = q[j] - 16 * g;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                unsigned v = 0;
                if (bytes >= 4) {                          // the same for every lane
                    const int from = min(at + 4 * d, bytes - 4);
                    __builtin_memcpy(&v, row + from, 4);
                    v >>= 8 * ((at + 4 * d - from) & 3);
                } else if (at + 4 * d == 0) {
                    for (int b = 0; b < bytes; ++b) v |= (unsigned)row[b] << (8 * b);
                }
                w.q[j][d] = v;
            }
        }
    }
};

// A step's products: x(t, slice) gives row tile t's fragment of a slice,
// reordered; scales and zeros point at the step's first group of the lane's first
// column, `pitch` values to a column.
template <int FMT, int MT, int SLICES, bool ZEROS, int PITCH, int J, typename X>
__device__ __forceinline__ void multiply(Weights<J>& w, const uint16_t* scales, const uint16_t* zeros, X&& x_at,
                                         floatx4 (&acc)[MT][J]) {
    using D = W4<FMT>;
    const floatx4 zero4 = {0.f, 0.f, 0.f, 0.f};
    const u32x4 ones = {D::ONES, D::ONES, D::ONES, D::ONES};
    unsigned mask = D::MASK, base = D::BASE;
    asm("" : "+s"(mask));
    asm("" : "+v"(base));
#pragma unroll
    for (int j = 0; j < J; ++j) transpose_groups(w.q[j]);
#pragma unroll
    for (int i = 0; i < 4 / SLICES; ++i) {
        floatx4 sum[MT][J], sx[MT];
#pragma unroll
        for (int h = 0; h < SLICES; ++h) {
            const int slice = i * SLICES + h;
            u32x4 v[J];
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = D::expand(w.q[j][slice], mask, base);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const u32x4 x = x_at(t, slice);
                sx[t] = mfma16x16<FMT>(x, ones, h == 0 ? zero4 : sx[t]);
#pragma unroll
                for (int j = 0; j < J; ++j) sum[t][j] = mfma16x16<FMT>(x, v[j], h == 0 ? zero4 : sum[t][j]);
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float s = D::value(scales[16 * j * PITCH + i]);
            const float z = 16.0f + (ZEROS ? D::value(zeros[16 * j * PITCH + i]) : 8.0f);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[t][j][r] = __builtin_fmaf(s, __builtin_fmaf(-z, sx[t][r], sum[t][j][r]), acc[t][j][r]);
        }
    }
}

// Rows row .. of a block's sums through the epilogue, or to its plane.
__device__ __forceinline__ void finish_run(const W4Args& p, const EpilogueArgs& e, float* planes, int row, int col, floatx4 sum) {
    float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    if (planes != nullptr) {
        store_values<2>(planes, ((int64_t)blockIdx.z * p.M + row) * p.N + col, p.N - col, v);
        return;
    }
    EpilogueRun<4, false> run;
    float bias[4];
    load_bias(e, col, bias);
    run.load(e, row, col);
    run.finish(e, row, col, bias, v);
}

// The chunks of steps whose scales lie in LDS at a time, and what a block takes:
// block z along K whole steps from z block_steps on, the last one also the step
// across K, if there is one.  chunk(first, last, group) runs behind the barrier
// after which LDS holds the groups from `group` on of the steps first .. last - 1.
template <int SLICES, bool ZEROS, int COLS, int GROUPS, typename C, typename F>
__device__ __forceinline__ void for_chunks(const W4Args& p, const C& columns, int n0, int block_steps,
                                           GroupValues<COLS, GROUPS>& scales, GroupValues<COLS, GROUPS>* zeros, F&& chunk) {
    constexpr int STEPS = GROUPS / (4 / SLICES);
    const int whole = p.K / kStep, groups = ceil_div(p.K, p.group);
    const int begin = min((int)blockIdx.z * block_steps, whole);
    const int end = blockIdx.z == gridDim.z - 1 ? ceil_div(p.K, kStep) : min(begin + block_steps, whole);
    for (int first = begin; first < end; first += STEPS) {
        const int last = min(first + STEPS, end), group = columns.group_of(first);
        const int count = min(columns.group_of(last - 1) + 4 / SLICES, groups) - group;
        if (first != begin) __syncthreads();               // the chunk before is read
        scales.fill(p.scales, p.ld_scales, n0, p.N, group, count, groups);
        if constexpr (ZEROS) zeros->fill(p.zeros, p.ld_zeros, n0, p.N, group, count, groups);
        __syncthreads();
        chunk(first, last, group);
    }
}

// 16 rows, J tiles of 16 columns, WAVES waves along K, two steps in flight.
template <int FMT, int J, int WAVES, int SLICES, bool ZEROS>
__global__ __launch_bounds__(64 * WAVES)
void linear_w4_kernel(W4Args p, EpilogueArgs e, int block_steps, float* planes) {
    constexpr int COLS = 16 * J, ROWS = 16, PITCH = COLS + 4, GROUPS = 128;
    using Values = GroupValues<COLS, GROUPS>;
    __shared__ __attribute__((aligned(16))) float part[WAVES][ROWS][PITCH];
    __shared__ __attribute__((aligned(16))) Values values[ZEROS ? 2 : 1];
    using D = W4<FMT>;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n0 = COLS * (int)blockIdx.x, m0 = ROWS * (int)blockIdx.y;
    const uint16_t* const xrow = p.X + (int64_t)min(m0 + c, p.M - 1) * p.ldx;
    const Columns<J, SLICES> columns(p, n0, lane);
    struct Step {
        u32x4 x[4];
        Weights<J> w;
    };
    auto load = [&](Step& st, int step) __attribute__((always_inline)) {
        columns.load(st.w, step);
#pragma unroll
        for (int i = 0; i < 4; ++i) __builtin_memcpy(&st.x[i], xrow + step * kStep + 8 * g + 32 * i, 16);
    };
    floatx4 acc[1][J];
#pragma unroll
    for (int j = 0; j < J; ++j) acc[0][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int whole = p.K / kStep;
    auto chunk = [&](int first, int last, int group) __attribute__((always_inline)) {
        const int count = min(last, whole) - first;
        const int begin = first + count * wave / WAVES, end = first + count * (wave + 1) / WAVES;
        auto compute = [&](Step& st, int step) __attribute__((always_inline)) {
            const int at = columns.group_of(step) - group;
            multiply<FMT, 1, SLICES, ZEROS, Values::PITCH>(
                st.w, &values[0].v[c][at], &values[ZEROS ? 1 : 0].v[c][at],
                [&](int, int slice) __attribute__((always_inline)) { return D::reorder(st.x[slice]); }, acc);
        };
        // No branch around the loads (the wait for one step's would otherwise wait
        // for both), so an odd number of steps loads the last one twice.
        if (begin < end) {
            Step s0, s1;
            load(s0, begin);
            load(s1, min(begin + 1, end - 1));
            int i = begin;
            for (; i + 2 < end; i += 2) {
                compute(s0, i);
                load(s0, i + 2);
                __builtin_amdgcn_sched_barrier(0);
                compute(s1, i + 1);
                load(s1, min(i + 3, end - 1));
                __builtin_amdgcn_sched_barrier(0);
            }
            compute(s0, i);
            if (i + 1 < end) compute(s1, i + 1);
        }
        if (last > whole && wave == WAVES - 1) {           // the step across K
            Step st;
            columns.load_last(st.w, p.K, whole);
#pragma unroll
            for (int i = 0; i < 4; ++i) st.x[i] = load_edge(xrow, whole * kStep + 8 * g + 32 * i, p.K);
            compute(st, whole);
        }
    };
    for_chunks<SLICES, ZEROS>(p, columns, n0, block_steps, values[0], values + (ZEROS ? 1 : 0), chunk);
    // Register r of acc[j]: row 4 g + r, column 16 j + c.
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][4 * g + r][16 * j + c] = acc[0][j][r];
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * COLS / 4; i += 64 * WAVES) {
        const int row = i / (COLS / 4), tc = 4 * (i % (COLS / 4)), col = n0 + tc;
        if (m0 + row >= p.M || col >= p.N) continue;
        floatx4 s = *reinterpret_cast<const floatx4*>(&part[0][row][tc]);
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += *reinterpret_cast<const floatx4*>(&part[w][row][tc]);
        finish_run(p, e, planes, m0 + row, col, s);
    }
}

// 16 MT rows x 128 columns: four waves of 32 columns share x's step through one
// of two stages of LDS, a row of 128 k as 16 runs of 8, run r at place r ^ (row %
// 16) (the 16 rows that a read takes then lie on all banks), reordered on the
// way in.  The next step's x and weights are in flight.
template <int FMT, int MT, int SLICES, bool ZEROS>
__global__ __launch_bounds__(256, 2)
void linear_w4_tile_kernel(W4Args p, EpilogueArgs e, int block_steps, float* planes) {
    constexpr int ROWS = 16 * MT, J = 2, RUNS = ROWS * 16 / 256, PITCH = 36, GROUPS = 64;
    using Values = GroupValues<128, GROUPS>;
    __shared__ __attribute__((aligned(16))) u32x4 stages[2][ROWS * 16];
    __shared__ __attribute__((aligned(16))) Values values[ZEROS ? 2 : 1];
    static_assert(sizeof(stages) >= 4 * 16 * PITCH * 4, "the epilogue's patches fit");
    using D = W4<FMT>;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n0 = 128 * (int)blockIdx.x + 32 * wave, m0 = ROWS * (int)blockIdx.y;
    const Columns<J, SLICES> columns(p, n0, lane);
    // This thread's runs of a step of x: run threadIdx.x % 16 of rows
    // threadIdx.x / 16 + 16 i.
    const int run = threadIdx.x & 15, row = threadIdx.x >> 4;
    const uint16_t* xrow[RUNS];
#pragma unroll
    for (int i = 0; i < RUNS; ++i) xrow[i] = p.X + (int64_t)min(m0 + row + 16 * i, p.M - 1) * p.ldx;
    u32x4 x[RUNS];
    auto load_x = [&](int step) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < RUNS; ++i) __builtin_memcpy(&x[i], xrow[i] + step * kStep + 8 * run, 16);
    };
    floatx4 acc[MT][J];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < J; ++j) acc[t][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    // x's step into a stage, whose readers, two steps ago, passed the last barrier;
    // then everyone's is there.
    auto share_x = [&](u32x4* stage) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < RUNS; ++r) stage[16 * (row + 16 * r) + (run ^ row)] = D::reorder(x[r]);
    };
    auto arrive = [&]() __attribute__((always_inline)) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    const int whole = p.K / kStep;
    auto chunk = [&](int first, int last, int group) __attribute__((always_inline)) {
        const int end = min(last, whole);
        auto compute = [&](Weights<J>& w, int step, const u32x4* stage) __attribute__((always_inline)) {
            const int at = columns.group_of(step) - group;
            multiply<FMT, MT, SLICES, ZEROS, Values::PITCH>(
                w, &values[0].v[32 * wave + c][at], &values[ZEROS ? 1 : 0].v[32 * wave + c][at],
                [&](int t, int slice) __attribute__((always_inline)) { return stage[16 * (16 * t + c) + ((4 * slice + g) ^ c)]; },
                acc);
        };
        if (first < end) {
            Weights<J> w0, w1;
            load_x(first);
            columns.load(w0, first);
            columns.load(w1, min(first + 1, end - 1));
            for (int i = first; i < end; i += 2) {
                share_x(stages[0]);
                load_x(min(i + 1, end - 1));
                arrive();
                compute(w0, i, stages[0]);
                columns.load(w0, min(i + 2, end - 1));
                if (i + 1 >= end) break;
                share_x(stages[1]);
                load_x(min(i + 2, end - 1));
                arrive();
                compute(w1, i + 1, stages[1]);
                columns.load(w1, min(i + 3, end - 1));
            }
        }
        if (last > whole) {                                // the step across K
            Weights<J> w;
            columns.load_last(w, p.K, whole);
#pragma unroll
            for (int i = 0; i < RUNS; ++i) x[i] = load_edge(xrow[i], whole * kStep + 8 * run, p.K);
            __syncthreads();                               // both stages are read
            share_x(stages[0]);
            arrive();
            compute(w, whole, stages[0]);
        }
    };
    for_chunks<SLICES, ZEROS>(p, columns, n0 - 32 * wave, block_steps, values[0], values + (ZEROS ? 1 : 0), chunk);
    __syncthreads();                                       // the stages are read
    // 16 rows at a time through the wave's patch, a run of 4 columns to a lane.
    float* const patch = reinterpret_cast<float*>(stages) + wave * 16 * PITCH;
    const int col = n0 + 4 * (lane & 7);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) patch[(4 * g + r) * PITCH + 16 * j + c] = acc[t][j][r];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = 8 * h + (lane >> 3), out = m0 + 16 * t + at;
            const floatx4 s = *reinterpret_cast<const floatx4*>(patch + at * PITCH + 4 * (lane & 7));
            if (out < p.M && col < p.N) finish_run(p, e, planes, out, col, s);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

// ------------------------------------------------------- choice of kernel

struct Plan {
    int rows, cols;                    // of a block
    int splits, block_steps;           // blocks along K; whole steps of each
};

// Up to 16 rows: 16 columns on eight waves, or 32 on four where they make a block
// for every CU and more (1 x 8192 x 8192 13.6 us in a graph against 14.2, 16 rows
// 17.6 against 24.2; 4096 x 4096 7.4 against 8.4).  Few columns with a long K
// split it over blocks, at 0.9 us a step of a wave and 4 for the pass (1 x 256 x
// 16384 8 us against 12).  More rows: blocks of 128 columns, K split until they
// make one for every CU (32 x 8192 x 8192 22 us with four shares, 52 with one; 64 x
// 4096 x 4096 15.5 with eight, 39 with one).
Plan make_plan(int M, int N, int K) {
    Plan q{};
    const int steps = K / kStep;
    int splits = 1;
    if (M <= 16) {
        q.rows = 16;
        q.cols = N >= 32 * 256 ? 32 : 16;
        const int blocks = ceil_div(N, q.cols);
        double least = 1e30;
        for (int s = 1; s <= 16 && (s == 1 || blocks * s <= 128); s *= 2) {
            const double t = 0.9 * ceil_div(steps, 8 * s) + (s > 1 ? 4.0 : 0.0);
            if (t < least) {
                least = t;
                splits = s;
            }
        }
    } else {
        q.rows = M <= 32 ? 32 : 64;
        q.cols = 128;
        const int64_t blocks = (int64_t)ceil_div(N, 128) * ceil_div(M, q.rows);
        splits = blocks >= 256 ? 1 : (int)(256 / blocks);
        if (splits > 32) splits = 32;
        if (splits > steps / 2) splits = steps / 2;
        if (splits < 1) splits = 1;
    }
    q.block_steps = steps > splits ? ceil_div(steps, splits) : 1;
    q.splits = steps > 0 ? ceil_div(steps, q.block_steps) : 1;
    return q;
}

template <int FMT, int SLICES, bool ZEROS>
void launch(const W4Args& p, const EpilogueArgs& e, hipStream_t s, const Plan& q, float* planes) {
    const dim3 grid(ceil_div(p.N, q.cols), ceil_div(p.M, q.rows), q.splits);
    const int n = q.block_steps;
    if (q.rows == 64)
        hipLaunchKernelGGL((linear_w4_tile_kernel<FMT, 4, SLICES, ZEROS>), grid, dim3(256), 0, s, p, e, n, planes);
    else if (q.rows == 32)
        hipLaunchKernelGGL((linear_w4_tile_kernel<FMT, 2, SLICES, ZEROS>), grid, dim3(256), 0, s, p, e, n, planes);
    else if (q.cols == 32)
        hipLaunchKernelGGL((linear_w4_kernel<FMT, 2, 4, SLICES, ZEROS>), grid, dim3(256), 0, s, p, e, n, planes);
    else
        hipLaunchKernelGGL((linear_w4_kernel<FMT, 1, 8, SLICES, ZEROS>), grid, dim3(512), 0, s, p, e, n, planes);
}

template <int FMT, bool ZEROS>
void launch_groups(const W4Args& p, const EpilogueArgs& e, hipStream_t s, const Plan& q, float* planes) {
    if (p.group == 32) launch<FMT, 1, ZEROS>(p, e, s, q, planes);
    else if (p.group == 64) launch<FMT, 2, ZEROS>(p, e, s, q, planes);
    else launch<FMT, 4, ZEROS>(p, e, s, q, planes);
}

}  // namespace

int64_t linear_w4_workspace(int M, int N, int K) {
    const Plan q = make_plan(M, N, K);
    return q.splits > 1 ? 4 * (int64_t)q.splits * M * N : 0;
}

hipError_t launch_linear_w4(const W4Args& p, const EpilogueArgs& e, hipStream_t s, int format, void* workspace) {
    const Plan q = make_plan(p.M, p.N, p.K);
    float* const planes = q.splits > 1 ? static_cast<float*>(workspace) : nullptr;
    if (format == 0 && p.zeros != nullptr) launch_groups<0, true>(p, e, s, q, planes);
    else if (format == 0) launch_groups<0, false>(p, e, s, q, planes);
    else if (p.zeros != nullptr) launch_groups<1, true>(p, e, s, q, planes);
    else launch_groups<1, false>(p, e, s, q, planes);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || planes == nullptr) return err;
    return launch_epilogue_pass(e, 2, planes, p.N, q.splits, (int64_t)p.M * p.N, nullptr, s);
}

}  // namespace gemmf32
