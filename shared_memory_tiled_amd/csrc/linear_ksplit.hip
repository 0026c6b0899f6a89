// linear_ksplit.hip -- the product with its epilogue on 64 x 64 tiles whose
// four waves split K (KsplitCore): runs of 4 columns, what the epilogue reads
// loaded before the partial tiles are added.
//
// Built with the matrix instructions' vector-register form, as
// mfma16_ksplit.hip.
#include "epilogue.h"
#include "linear_kernels.h"
#include "mfma16_ksplit_core.h"

namespace gemmf32 {

namespace {

template <int FMT, bool KCA, bool KCB, bool GRADIENT>
__global__ __launch_bounds__(256)
void linear_ksplit_kernel(Gemm16Args p, EpilogueArgs e, int tiles_m, int tiles_n, int group_m, float* partials) {
    using Core = KsplitCore<FMT, KCA, KCB>;
    __shared__ __attribute__((aligned(16))) uint16_t lds[Core::LDS_ELEMS];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int tm, tn;
    grouped_tile((int)blockIdx.x, tiles_m, tiles_n, group_m, &tm, &tn);
    const int m0 = tm * 64, n0 = tn * 64;
    const int col = n0 + Core::sum_col(lane);
    Core::run(p, m0, n0, lds);
    float bias[4];
    if constexpr (!GRADIENT) load_bias(e, col, bias);
    EpilogueRun<4, GRADIENT> run[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int row = m0 + Core::sum_row(w, lane, it);
        if (row < e.M && col < e.N) run[it].load(e, row, col);
    }
    float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int row = m0 + Core::sum_row(w, lane, it);
        if (row >= e.M || col >= e.N) continue;
        const floatx4 s = Core::sum4(lds, w, lane, it);
        float v[4] = {s[0], s[1], s[2], s[3]};
        run[it].finish(e, row, col, bias, v);
        if constexpr (GRADIENT) {
#pragma unroll
            for (int c = 0; c < 4; ++c) sums[c] += v[c];
        }
    }
    if constexpr (GRADIENT) {
        if (partials == nullptr) return;                  // the same for every thread
        float* const part = reinterpret_cast<float*>(lds);
        __syncthreads();                                  // the partial tiles are read
#pragma unroll
        for (int c = 0; c < 4; ++c) {                     // lanes 4 apart within 16 hold other rows
            float s = sums[c];
            s += __shfl_xor(s, 4, 64);
            s += __shfl_xor(s, 8, 64);
            if ((lane & 12) == 0) part[64 * w + Core::sum_col(lane) + c] = s;
        }
        __syncthreads();
        const int c = threadIdx.x;
        if (c < 64 && n0 + c < e.N)
            partials[(int64_t)tm * e.N + n0 + c] = ((part[c] + part[64 + c]) + part[128 + c]) + part[192 + c];
    }
}

// K split over blocks too: block (tile, y) takes k = y k_share .. (a multiple
// of 64) and stores its sums as plane y of M x N floats.
template <int FMT, bool KCA, bool KCB>
__global__ __launch_bounds__(256)
void linear_ksplit_planes_kernel(Gemm16Args p, int M, int N, int k_share, int tiles_m, int tiles_n, int group_m,
                                 float* planes) {
    using Core = KsplitCore<FMT, KCA, KCB>;
    __shared__ __attribute__((aligned(16))) uint16_t lds[Core::LDS_ELEMS];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int tm, tn;
    grouped_tile((int)blockIdx.x, tiles_m, tiles_n, group_m, &tm, &tn);
    const int m0 = tm * 64, n0 = tn * 64;
    const int k0 = (int)blockIdx.y * k_share;
    p.A += KCA ? (int64_t)k0 : k0 * p.lda;
    p.B += KCB ? (int64_t)k0 : k0 * p.ldb;
    p.K = min(p.K - k0, k_share);
    Core::run(p, m0, n0, lds);
    const int col = n0 + Core::sum_col(lane);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int row = m0 + Core::sum_row(w, lane, it);
        if (row >= M || col >= N) continue;
        const floatx4 s = Core::sum4(lds, w, lane, it);
        const float v[4] = {s[0], s[1], s[2], s[3]};
        store_values<2>(planes, ((int64_t)blockIdx.y * M + row) * N + col, N - col, v);
    }
}

template <int FMT, bool KCA, bool KCB>
void launch_planes(const Gemm16Args& p, int M, int N, hipStream_t s, int tm, int tn, int k_share, float* planes) {
    constexpr int kGroupM = 8;
    hipLaunchKernelGGL((linear_ksplit_planes_kernel<FMT, KCA, KCB>), dim3((unsigned)(tm * tn), ceil_div(p.K, k_share)),
                       dim3(256), 0, s, p, M, N, k_share, tm, tn, kGroupM, planes);
}

template <int FMT, bool KCA, bool KCB>
void launch(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int tm, int tn, float* partials) {
    constexpr int kGroupM = 8;                            // as gemm_mixed's launches of these tiles
    const dim3 g((unsigned)(tm * tn)), b(256);
    if (e.gradient)
        hipLaunchKernelGGL((linear_ksplit_kernel<FMT, KCA, KCB, true>), g, b, 0, s, p, e, tm, tn, kGroupM, partials);
    else
        hipLaunchKernelGGL((linear_ksplit_kernel<FMT, KCA, KCB, false>), g, b, 0, s, p, e, tm, tn, kGroupM, partials);
}

}  // namespace

hipError_t launch_linear_ksplit(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                                int op_b, float* partials) {
    const int tm = ceil_div(p.M, 64), tn = ceil_div(p.N, 64);
    if ((int64_t)tm * tn > 0x7FFFFFFFll / 256) return hipErrorInvalidValue;
    switch (4 * (format ? 1 : 0) + 2 * (op_a ? 1 : 0) + (op_b ? 1 : 0)) {
        case 0: launch<0, true, false>(p, e, s, tm, tn, partials); break;
        case 1: launch<0, true, true>(p, e, s, tm, tn, partials); break;
        case 2: launch<0, false, false>(p, e, s, tm, tn, partials); break;
        case 3: launch<0, false, true>(p, e, s, tm, tn, partials); break;
        case 4: launch<1, true, false>(p, e, s, tm, tn, partials); break;
        case 5: launch<1, true, true>(p, e, s, tm, tn, partials); break;
        case 6: launch<1, false, false>(p, e, s, tm, tn, partials); break;
        default: launch<1, false, true>(p, e, s, tm, tn, partials); break;
    }
    return hipGetLastError();
}

hipError_t launch_linear_ksplit_planes(const Gemm16Args& p, int M, int N, hipStream_t s, int format, int op_a, int op_b,
                                       int k_share, float* planes) {
    const int tm = ceil_div(M, 64), tn = ceil_div(N, 64);
    switch (4 * (format ? 1 : 0) + 2 * (op_a ? 1 : 0) + (op_b ? 1 : 0)) {
        case 0: launch_planes<0, true, false>(p, M, N, s, tm, tn, k_share, planes); break;
        case 1: launch_planes<0, true, true>(p, M, N, s, tm, tn, k_share, planes); break;
        case 2: launch_planes<0, false, false>(p, M, N, s, tm, tn, k_share, planes); break;
        case 3: launch_planes<0, false, true>(p, M, N, s, tm, tn, k_share, planes); break;
        case 4: launch_planes<1, true, false>(p, M, N, s, tm, tn, k_share, planes); break;
        case 5: launch_planes<1, true, true>(p, M, N, s, tm, tn, k_share, planes); break;
        case 6: launch_planes<1, false, false>(p, M, N, s, tm, tn, k_share, planes); break;
        default: launch_planes<1, false, true>(p, M, N, s, tm, tn, k_share, planes); break;
    }
    return hipGetLastError();
}

}  // namespace gemmf32
