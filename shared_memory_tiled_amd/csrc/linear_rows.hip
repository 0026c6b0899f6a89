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

hipError_t launch_linear_rows(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_b,
                              int splits, float* planes) {
    if (format == 0 && op_b) launch_tiles<0, true>(p, e, s, splits, planes);
    else if (format == 0) launch_tiles<0, false>(p, e, s, splits, planes);
    else if (op_b) launch_tiles<1, true>(p, e, s, splits, planes);
    else launch_tiles<1, false>(p, e, s, splits, planes);
    return hipGetLastError();
}

}  // namespace gemmf32
