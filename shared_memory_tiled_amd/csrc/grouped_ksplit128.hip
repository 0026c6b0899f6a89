// grouped_ksplit128.hip -- the grouped layer on 128 x 128 tiles whose four waves
// split K (Ksplit128Core): runs of 4 columns, a round of what the epilogue reads
// loaded ahead of the exchange.
#include "grouped_tiles.h"
#include "mfma16_ksplit128_core.h"

namespace gemmf32 {

namespace {

template <typename Core>
__device__ __forceinline__ void finish(const floatx4 (&acc)[8][8], const EpilogueArgs& e, int m0, int n0,
                                       unsigned char* lds) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = n0 + 4 * (lane & 31);
    float bias[4];
    load_bias(e, col, bias);
    EpilogueRun<4, false> run[8];
    auto load = [&](int a, int it) __attribute__((always_inline)) {
        const int row = m0 + 16 * (4 * a + w) + 2 * it + (lane >> 5);
        if (row < e.M && col < e.N) run[it].load(e, row, col);
    };
#pragma unroll
    for (int it = 0; it < 8; ++it) load(0, it);
    Core::exchange(
        acc, lds,
        [&](int a, int it, int r, int, floatx4 sum, float*) __attribute__((always_inline)) {
            float v[4] = {sum[0], sum[1], sum[2], sum[3]};
            if (m0 + r < e.M && col < e.N) run[it].finish(e, m0 + r, col, bias, v);
            if (a == 0) load(1, it);
        },
        [](int) {});
}

template <int FMT, bool KCB>
__global__ __launch_bounds__(256)
void grouped_ksplit128_kernel(GroupedArgs a, Gemm16Args p, EpilogueArgs e, int tiles_n, int group_m) {
    using Core = Ksplit128Core<FMT, true, KCB>;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Core::LDS_BYTES];
    const GroupRows r = locate_group_tile<128>(a, (int)blockIdx.x, tiles_n, group_m);
    if (r.rows < 0) return;
    enter_group(a, r, &p, &e);
    const int m0 = 128 * r.tm, n0 = 128 * r.tn;
    p.A += (int64_t)m0 * p.lda;
    p.M = min(r.rows - m0, 128);
    floatx4 acc[8][8];
    Core::run(p, 0, n0, lds, acc);
    GEMM16_PIN_ACCUMULATORS(acc, 8, 8);
    finish<Core>(acc, e, m0, n0, lds);
}

template <int FMT>
__global__ __launch_bounds__(256)
void grouped_grad_ksplit128_kernel(GroupedArgs a, Gemm16Args p, EpilogueArgs e, int tiles_m, int tiles_n, int group_m) {
    using Core = Ksplit128Core<FMT, false, false>;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Core::LDS_BYTES];
    const GroupRows r = locate_grad_tile(a, (int)blockIdx.x, tiles_m, tiles_n, group_m);
    enter_grad_group(a, r, &p, &e);
    const int m0 = 128 * r.tm, n0 = 128 * r.tn;
    if (r.rows == 0) return zero_tile<128>(e, m0, n0);
    floatx4 acc[8][8];
    Core::run(p, m0, n0, lds, acc);
    GEMM16_PIN_ACCUMULATORS(acc, 8, 8);
    finish<Core>(acc, e, m0, n0, lds);
}

}  // namespace

hipError_t launch_grouped_ksplit128(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                                    int format, int op_b) {
    constexpr int kGroupM = 8;
    const int tn = ceil_div(p.N, 128);
    const dim3 g((unsigned)(grouped_row_tiles(a.rows, a.groups, 128) * tn)), b(256);
    if (format == 0 && op_b) hipLaunchKernelGGL((grouped_ksplit128_kernel<0, true>), g, b, 0, s, a, p, e, tn, kGroupM);
    else if (format == 0) hipLaunchKernelGGL((grouped_ksplit128_kernel<0, false>), g, b, 0, s, a, p, e, tn, kGroupM);
    else if (op_b) hipLaunchKernelGGL((grouped_ksplit128_kernel<1, true>), g, b, 0, s, a, p, e, tn, kGroupM);
    else hipLaunchKernelGGL((grouped_ksplit128_kernel<1, false>), g, b, 0, s, a, p, e, tn, kGroupM);
    return hipGetLastError();
}

hipError_t launch_grouped_grad_ksplit128(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e,
                                         hipStream_t s, int format) {
    constexpr int kGroupM = 8;
    const int tm = ceil_div(p.M, 128), tn = ceil_div(p.N, 128);
    const dim3 g((unsigned)(tm * tn * a.groups)), b(256);
    if (format == 0) hipLaunchKernelGGL((grouped_grad_ksplit128_kernel<0>), g, b, 0, s, a, p, e, tm, tn, kGroupM);
    else hipLaunchKernelGGL((grouped_grad_ksplit128_kernel<1>), g, b, 0, s, a, p, e, tm, tn, kGroupM);
    return hipGetLastError();
}

}  // namespace gemmf32
