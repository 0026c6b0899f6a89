// linear_rows.hip -- the product with its epilogue for few rows (a decoder's
// tokens): M <= 64, where the weight is read once and its bytes set the time.
//
// Blocks of four waves take 128 columns and a share of K, each wave a quarter
// of it in 32-deep steps (consecutive ones: with the weight stored N x K two
// steps share a cache line).  A step is 8 matrix instructions
// v_mfma_f32_16x16x32 per 16 rows of X, straight from registers: X's fragment
// (lane l: row l % 16, k 8 (l / 16) .. + 7) and, for instruction j, the weight's
// column 8 (l % 16) + j of the block.  With the weight stored N x K that is one
// 16-byte load per column and lane.  Stored K x N, a lane loads 8 rows of 8
// columns (16 lanes: 256 bytes of a row) and turns the 8 x 8 values in
// registers (32 v_perm_b32 per 8 KB of weight and wave, an eighth of the time
// in which a CU's share of memory bandwidth brings them).
//
// Nothing is staged in LDS before the end: each wave's loads of a step are in
// flight while it computes the step before, and a few waves per SIMD cover
// the memory latency.  The four waves' sums meet in LDS and are added in wave
// order; with K split over blocks too (so that 128-column blocks fill the
// CUs) each block stores its plane of sums and the epilogue pass adds them in
// order.  Columns past N and rows past M repeat the last one and are not
// stored; k past K loads as zero.
#include "epilogue.h"
#include "linear_kernels.h"
#include "mfma16_common.h"

namespace gemmf32 {

namespace {

constexpr int kCols = 128, kStep = 32, kWaves = 4;

// Eight consecutive 16-bit values from p, of which `valid` exist.
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int valid) {
    u32x4 v = {0, 0, 0, 0};
    if (valid >= 8) {
        __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) v[e / 2] |= (unsigned)p[e] << (16 * (e % 2));
    }
    return v;
}

template <int FMT, bool TB, int MT, bool FUSED>
__global__ __launch_bounds__(256)
void linear_rows_kernel(Gemm16Args p, EpilogueArgs e, int k_per_split, float* planes) {
    constexpr int PITCH = kCols + 4;
    __shared__ __attribute__((aligned(16))) float part[kWaves][16 * MT][PITCH];
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n0 = blockIdx.x * kCols;
    // The block's share of K, a quarter of it (whole steps) for each wave.
    const int share = k_per_split / kWaves;                 // k_per_split: a multiple of kWaves kStep
    const int k_begin = (int)blockIdx.y * k_per_split + wave * share;
    const int k_end = min(p.K, k_begin + share);

    struct Step {
        u32x4 x[MT], w[8];
    };
    const uint16_t* xrow[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xrow[t] = p.A + (int64_t)min(16 * t + c, p.M - 1) * p.lda;
    // Columns as loaded: those past N repeat others, and a chunk across N reads
    // on into the next row -- unless there is none, or rows are too short for
    // it to be the next one.
    const bool inside = n0 + kCols <= p.N;                  // the block's columns all exist
    const int whole_k = inside ? p.K : p.ldb >= 8 ? p.K - 1 : 0;   // rows below it load whole chunks
    const uint16_t* wcol[TB ? 8 : 1];
    if constexpr (TB) {
#pragma unroll
        for (int j = 0; j < 8; ++j) wcol[j] = p.B + (int64_t)min(n0 + 8 * c + j, p.N - 1) * p.ldb;
    } else {
        wcol[0] = p.B + (n0 + 8 * c < p.N ? n0 + 8 * c : 0);
    }
    auto load = [&](Step& s, int k0) __attribute__((always_inline)) {
        const int k = k0 + 8 * g;
        if (k0 + kStep <= k_end && (TB || k0 + kStep <= whole_k)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint16_t* q = TB ? wcol[TB ? j : 0] + k : wcol[0] + (int64_t)(k + j) * p.ldb;
                __builtin_memcpy(&s.w[j], q, 16);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) __builtin_memcpy(&s.x[t], xrow[t] + k, 16);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (TB)
                    s.w[j] = load8(wcol[j] + k, k_end - k);
                else
                    s.w[j] = load8(p.B + (int64_t)(k + j) * p.ldb + n0 + 8 * c, k + j < k_end ? p.N - (n0 + 8 * c) : 0);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) s.x[t] = load8(xrow[t] + k, k_end - k);
        }
    };
    floatx4 acc[MT][8];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const Step& s) __attribute__((always_inline)) {
        u32x4 b[8];
        if constexpr (TB) {
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = s.w[j];
        } else {                                            // rows of columns -> columns of rows
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const unsigned lo = s.w[2 * r][q], hi = s.w[2 * r + 1][q];
                    b[2 * q][r] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
                    b[2 * q + 1][r] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
                }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[t][j] = mfma16x16<FMT>(s.x[t], b[j], acc[t][j]);
    };
    int k0 = k_begin;
    if (k0 < k_end) {
        Step s0, s1;
        load(s0, k0);
        for (;;) {
            const int k1 = k0 + kStep, k2 = k1 + kStep;
            if (k1 < k_end) load(s1, k1);
            compute(s0);
            if (k1 >= k_end) break;
            if (k2 < k_end) load(s0, k2);
            compute(s1);
            if (k2 >= k_end) break;
            k0 = k2;
        }
    }

    // Register r of acc[t][j]: row 16 t + 4 g + r, column 8 c + j.
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            floatx4* q = reinterpret_cast<floatx4*>(&part[wave][16 * t + 4 * g + r][8 * c]);
            q[0] = floatx4{acc[t][0][r], acc[t][1][r], acc[t][2][r], acc[t][3][r]};
            q[1] = floatx4{acc[t][4][r], acc[t][5][r], acc[t][6][r], acc[t][7][r]};
        }
    __syncthreads();
    const int tc = 4 * (threadIdx.x & 31), col = n0 + tc;
    if (col >= p.N) return;
    float bias[4];
    if constexpr (FUSED) load_bias(e, col, bias);
    for (int row = threadIdx.x / 32; row < p.M; row += 8) {
        floatx4 s = *reinterpret_cast<const floatx4*>(&part[0][row][tc]);
#pragma unroll
        for (int u = 1; u < kWaves; ++u) s += *reinterpret_cast<const floatx4*>(&part[u][row][tc]);
        float v[4] = {s[0], s[1], s[2], s[3]};
        if constexpr (FUSED) {
            EpilogueRun<4, false> run;
            run.load(e, row, col);
            run.finish(e, row, col, bias, v);
        } else {
            store_values<2>(planes, ((int64_t)blockIdx.y * p.M + row) * p.N + col, p.N - col, v);
        }
    }
}

// The same without a second launch, for problems whose blocks of 128 columns
// would have to split K: blocks of sixteen waves take 32 columns and all of K,
// each wave a sixteenth of it, J = 2 columns per lane.  Stored K x N, a row's
// 32 columns are half a cache line; the block beside it, on the same XCD,
// reads the other half.  A CU alone brings 20 to 40 KB of weight per us this
// way, whatever is in flight (blocks of 64 columns, whole cache lines, take
// twice as long), so a long K is better split over more CUs.
constexpr int kFusedWaves = 16, kFusedCols = 32;
template <int FMT, bool TB, int MT>
__global__ __launch_bounds__(64 * kFusedWaves)
void linear_rows_fused_kernel(Gemm16Args p, EpilogueArgs e, int share) {
    constexpr int COLS = kFusedCols, J = COLS / 16, PITCH = COLS + 4, ROW_THREADS = COLS / 4;
    __shared__ __attribute__((aligned(16))) float part[kFusedWaves][16 * MT][PITCH];
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n0 = COLS * xcd_contiguous((int)blockIdx.x, (int)gridDim.x);
    const int k_begin = wave * share, k_end = min(p.K, k_begin + share);   // share: a multiple of kStep
    // what the epilogue reads: ROW_THREADS threads per row, four columns each
    const int row = threadIdx.x / ROW_THREADS, tc = 4 * (threadIdx.x % ROW_THREADS), col = n0 + tc;
    const bool stores = row < p.M && col < p.N;
    float bias[4];
    EpilogueRun<4, false> run;
    if (stores) {
        load_bias(e, col, bias);
        run.load(e, row, col);
    }

    struct Step {
        u32x4 x[MT];
        unsigned w[4 * J];                                  // TB: J columns of 8 k; else 8 rows of J columns
    };
    const uint16_t* xrow[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xrow[t] = p.A + (int64_t)min(16 * t + c, p.M - 1) * p.lda;
    // Columns across N read on into the next row, as above.
    const bool inside = n0 + COLS <= p.N;
    const int whole_k = inside ? p.K : p.ldb >= J ? p.K - 1 : 0;
    const int first = n0 + J * c;
    const uint16_t* wcol[TB ? J : 1];
    if constexpr (TB) {
#pragma unroll
        for (int j = 0; j < J; ++j) wcol[j] = p.B + (int64_t)min(first + j, p.N - 1) * p.ldb;
    } else {
        wcol[0] = p.B + (first < p.N ? first : 0);
    }
    auto load = [&](Step& s, int k0) __attribute__((always_inline)) {
        const int k = k0 + 8 * g;
        if constexpr (TB) {
#pragma unroll
            for (int j = 0; j < J; ++j) __builtin_memcpy(s.w + 4 * j, wcol[TB ? j : 0] + k, 16);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) __builtin_memcpy(s.w + J / 2 * j, wcol[0] + (int64_t)(k + j) * p.ldb, 2 * J);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) __builtin_memcpy(&s.x[t], xrow[t] + k, 16);
    };
    auto load_ragged = [&](Step& s, int k0) __attribute__((always_inline)) {
        const int k = k0 + 8 * g;
        if constexpr (TB) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const u32x4 v = load8(wcol[TB ? j : 0] + k, k_end - k);
#pragma unroll
                for (int i = 0; i < 4; ++i) s.w[4 * j + i] = v[i];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < J; i += 2) {
                    const uint16_t* const q = p.B + (int64_t)(k + j) * p.ldb + first + i;
                    s.w[J / 2 * j + i / 2] =
                        k + j < k_end && first + i < p.N
                            ? (unsigned)q[0] | (first + i + 1 < p.N ? (unsigned)q[1] << 16 : 0u) : 0u;
                }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) s.x[t] = load8(xrow[t] + k, k_end - k);
    };
    floatx4 acc[MT][J];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < J; ++j) acc[t][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const Step& s) __attribute__((always_inline)) {
        u32x4 b[J];
        if constexpr (TB) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) b[j][r] = s.w[4 * j + r];
        } else {                                            // rows of columns -> columns of rows
#pragma unroll
            for (int q = 0; q < J / 2; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const unsigned lo = s.w[J * r + q], hi = s.w[J * r + J / 2 + q];
                    b[2 * q][r] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
                    b[2 * q + 1][r] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
                }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < J; ++j) acc[t][j] = mfma16x16<FMT>(s.x[t], b[j], acc[t][j]);
    };
    // Whole steps, two in flight; the loop has no branch around its loads (the
    // wait for one step's would otherwise wait for both), so an odd number of
    // steps loads the last one twice.
    const int k_whole = min(k_end, TB ? p.K : whole_k);
    const int full = k_whole > k_begin ? (k_whole - k_begin) / kStep : 0;
    if (full > 0) {
        Step s0, s1;
        load(s0, k_begin);
        if (full > 1) load(s1, k_begin + kStep);
        int i = 0;
        for (; i + 2 < full; i += 2) {
            compute(s0);
            load(s0, k_begin + kStep * (i + 2));
            __builtin_amdgcn_sched_barrier(0);
            compute(s1);
            load(s1, k_begin + kStep * min(i + 3, full - 1));
            __builtin_amdgcn_sched_barrier(0);
        }
        compute(s0);
        if (i + 1 < full) compute(s1);
    }
    for (int k0 = k_begin + kStep * full; k0 < k_end; k0 += kStep) {
        Step s;
        load_ragged(s, k0);
        compute(s);
    }

    // Register r of acc[t][j]: row 16 t + 4 g + r, column J c + j.
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < J; ++j) part[wave][16 * t + 4 * g + r][J * c + j] = acc[t][j][r];
    __syncthreads();
    if (!stores) return;
    floatx4 s = *reinterpret_cast<const floatx4*>(&part[0][row][tc]);
#pragma unroll
    for (int u = 1; u < kFusedWaves; ++u) s += *reinterpret_cast<const floatx4*>(&part[u][row][tc]);
    float v[4] = {s[0], s[1], s[2], s[3]};
    run.finish(e, row, col, bias, v);
}

int steps_per_split(int K, int splits) { return ceil_div(ceil_div(K, kStep * kWaves), splits); }

template <int FMT, bool TB, int MT>
void launch_rows(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int splits, float* planes) {
    const int per = kStep * kWaves * steps_per_split(p.K, splits);
    const dim3 g(ceil_div(p.N, kCols), (unsigned)splits), b(256);
    if (planes == nullptr)
        hipLaunchKernelGGL((linear_rows_kernel<FMT, TB, MT, true>), g, b, 0, s, p, e, per, planes);
    else
        hipLaunchKernelGGL((linear_rows_kernel<FMT, TB, MT, false>), g, b, 0, s, p, e, per, planes);
}
template <int FMT, bool TB>
void launch_fused(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s) {
    const int share = kStep * ceil_div(ceil_div(p.K, kStep), kFusedWaves);
    const dim3 g(ceil_div(p.N, kFusedCols)), b(64 * kFusedWaves);
    if (p.M <= 16) hipLaunchKernelGGL((linear_rows_fused_kernel<FMT, TB, 1>), g, b, 0, s, p, e, share);
    else hipLaunchKernelGGL((linear_rows_fused_kernel<FMT, TB, 2>), g, b, 0, s, p, e, share);
}
template <int FMT, bool TB>
void launch_tiles(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int splits, float* planes) {
    if (p.M <= 16) launch_rows<FMT, TB, 1>(p, e, s, splits, planes);
    else if (p.M <= 32) launch_rows<FMT, TB, 2>(p, e, s, splits, planes);
    else launch_rows<FMT, TB, 4>(p, e, s, splits, planes);
}

}  // namespace

// One block per CU (24 x 8192 x 4096: 17 us with 256 blocks, 20 with 512 or
// 128), but at least two steps per wave, and no empty split.
int linear_rows_splits(int M, int N, int K) {
    const int blocks = ceil_div(N, kCols), steps = ceil_div(K, kStep * kWaves);
    int splits = 256 / blocks;
    if (splits > steps / 2) splits = steps / 2;
    if (splits < 1) return 1;
    return ceil_div(steps, steps_per_split(K, splits));
}

// Times of one row in a graph with a cold weight, fused against split, us
// (weight stored K x N, then N x K): 1024 x 1024 4.6 / 6.4, 4.7 / 7.4; 4096 x 1024
// (N x K) 4.9 / 7.0, 4.8 / 7.9; 2048 x 2048 6.2 / 7.3, 6.6 / 8.0; 8192 x 2048 10.6
// / 12.0; but 1024 x 4096 10.3 / 7.6, 10.5 / 8.5, 10000 x 1000 (more than one
// block per CU) 15.3 / 10.8, and 4096^2 17.0 / 12.9, 12.8 / 14.6 (16 rows 16.1 /
// 15.7), 6000^2 23.1 / 21.4, 20.7 / 25.2 (16 rows 27.7 / 26.5).  32 rows gain a
// little still (2048 x 2048 8.7 / 9.0).
bool linear_rows_fused(int M, int N, int K, int op_b) {
    if (M > 32 || N > 256 * kFusedCols) return false;
    return K <= 2048 || (op_b && M <= 8 && N >= 4096 && K <= 8192);
}

hipError_t launch_linear_rows_fused(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_b) {
    if (format == 0 && op_b) launch_fused<0, true>(p, e, s);
    else if (format == 0) launch_fused<0, false>(p, e, s);
    else if (op_b) launch_fused<1, true>(p, e, s);
    else launch_fused<1, false>(p, e, s);
    return hipGetLastError();
}

hipError_t launch_linear_rows(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_b,
                              int splits, float* planes) {
    if (format == 0 && op_b) launch_tiles<0, true>(p, e, s, splits, planes);
    else if (format == 0) launch_tiles<0, false>(p, e, s, splits, planes);
    else if (op_b) launch_tiles<1, true>(p, e, s, splits, planes);
    else launch_tiles<1, false>(p, e, s, splits, planes);
    return hipGetLastError();
}

}  // namespace gemmf32
