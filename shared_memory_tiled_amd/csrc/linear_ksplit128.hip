// linear_ksplit128.hip -- the product with its epilogue on 128 x 128 tiles
// whose four waves split K (Ksplit128Core): runs of 4 columns, a round of
// what the epilogue reads loaded ahead of the exchange.
#include "epilogue.h"
#include "linear_kernels.h"
#include "mfma16_ksplit128_core.h"
#include "mfma16_wide_core.h"

namespace gemmf32 {

namespace {

template <int FMT, bool KCA, bool KCB, bool GRADIENT>
__global__ __launch_bounds__(256)
void linear_ksplit128_kernel(Gemm16Args p, EpilogueArgs e, int tiles_m, int tiles_n, int group_m, float* partials) {
    using Core = Ksplit128Core<FMT, KCA, KCB>;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Core::LDS_BYTES];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int tm, tn;
    grouped_tile((int)blockIdx.x, tiles_m, tiles_n, group_m, &tm, &tn);
    const int m0 = tm * 128, n0 = tn * 128;
    const int col = n0 + 4 * (lane & 31);
    floatx4 acc[8][8];
    Core::run(p, m0, n0, lds, acc);
    GEMM16_PIN_ACCUMULATORS(acc, 8, 8);
    float bias[4];
    if constexpr (!GRADIENT) load_bias(e, col, bias);
    EpilogueRun<4, GRADIENT> run[8];
    auto load = [&](int a, int it) __attribute__((always_inline)) {
        const int row = m0 + 16 * (4 * a + w) + 2 * it + (lane >> 5);
        if (row < e.M && col < e.N) run[it].load(e, row, col);
    };
#pragma unroll
    for (int it = 0; it < 8; ++it) load(0, it);
    float sums[4] = {0.f, 0.f, 0.f, 0.f};
    Core::exchange(
        acc, lds,
        [&](int a, int it, int r, int, floatx4 sum, float*) __attribute__((always_inline)) {
            float v[4] = {sum[0], sum[1], sum[2], sum[3]};
            if (m0 + r < e.M && col < e.N) {
                run[it].finish(e, m0 + r, col, bias, v);
                if constexpr (GRADIENT) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) sums[c] += v[c];
                }
            }
            if (a == 0) load(1, it);
        },
        [](int) {});
    if constexpr (GRADIENT) {
        if (partials == nullptr) return;                  // the same for every thread
        float* const part = reinterpret_cast<float*>(lds);
        __syncthreads();                                  // the exchange is read
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float s = sums[c] + __shfl_xor(sums[c], 32, 64);
            if (lane < 32) part[128 * w + 4 * lane + c] = s;
        }
        __syncthreads();
        const int c = threadIdx.x;
        if (c < 128 && n0 + c < e.N)
            partials[(int64_t)tm * e.N + n0 + c] = ((part[c] + part[128 + c]) + part[256 + c]) + part[384 + c];
    }
}

template <int FMT, bool KCA, bool KCB>
void launch(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int tm, int tn, float* partials) {
    constexpr int kGroupM = 8;                            // as gemm_mixed's launches of these tiles
    const dim3 g((unsigned)(tm * tn)), b(256);
    if (e.gradient)
        hipLaunchKernelGGL((linear_ksplit128_kernel<FMT, KCA, KCB, true>), g, b, 0, s, p, e, tm, tn, kGroupM, partials);
    else
        hipLaunchKernelGGL((linear_ksplit128_kernel<FMT, KCA, KCB, false>), g, b, 0, s, p, e, tm, tn, kGroupM, partials);
}

}  // namespace

hipError_t launch_linear_ksplit128(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                                   int op_b, float* partials) {
    const int tm = ceil_div(p.M, 128), tn = ceil_div(p.N, 128);
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

}  // namespace gemmf32
