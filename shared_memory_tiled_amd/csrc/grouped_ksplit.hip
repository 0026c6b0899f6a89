// grouped_ksplit.hip -- the grouped layer on 64 x 64 tiles whose four waves
// split K (KsplitCore): runs of 4 columns, what the epilogue reads loaded before
// the partial tiles are added.
//
// Built with the matrix instructions' vector-register form, as
// mfma16_ksplit.hip.
#include "grouped_tiles.h"
#include "mfma16_ksplit_core.h"

namespace gemmf32 {

namespace {

template <typename Core>
__device__ __forceinline__ void finish(const EpilogueArgs& e, int m0, int n0, uint16_t* lds) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = n0 + Core::sum_col(lane);
    float bias[4];
    load_bias(e, col, bias);
    EpilogueRun<4, false> run[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int row = m0 + Core::sum_row(w, lane, it);
        if (row < e.M && col < e.N) run[it].load(e, row, col);
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int row = m0 + Core::sum_row(w, lane, it);
        if (row >= e.M || col >= e.N) continue;
        const floatx4 s = Core::sum4(lds, w, lane, it);
        float v[4] = {s[0], s[1], s[2], s[3]};
        run[it].finish(e, row, col, bias, v);
    }
}

template <int FMT, bool KCB>
__global__ __launch_bounds__(256)
void grouped_ksplit_kernel(GroupedArgs a, Gemm16Args p, EpilogueArgs e, int tiles_n, int group_m) {
    using Core = KsplitCore<FMT, true, KCB>;
    __shared__ __attribute__((aligned(16))) uint16_t lds[Core::LDS_ELEMS];
    const GroupRows r = locate_group_tile<64>(a, (int)blockIdx.x, tiles_n, group_m);
    if (r.rows < 0) return;
    enter_group(a, r, &p, &e);
    const int m0 = 64 * r.tm, n0 = 64 * r.tn;
    p.A += (int64_t)m0 * p.lda;
    p.M = min(r.rows - m0, 64);
    Core::run(p, 0, n0, lds);
    finish<Core>(e, m0, n0, lds);
}

template <int FMT>
__global__ __launch_bounds__(256)
void grouped_grad_ksplit_kernel(GroupedArgs a, Gemm16Args p, EpilogueArgs e, int tiles_m, int tiles_n, int group_m) {
    using Core = KsplitCore<FMT, false, false>;
    __shared__ __attribute__((aligned(16))) uint16_t lds[Core::LDS_ELEMS];
    const GroupRows r = locate_grad_tile(a, (int)blockIdx.x, tiles_m, tiles_n, group_m);
    enter_grad_group(a, r, &p, &e);
    const int m0 = 64 * r.tm, n0 = 64 * r.tn;
    if (r.rows == 0) return zero_tile<64>(e, m0, n0);
    Core::run(p, m0, n0, lds);
    finish<Core>(e, m0, n0, lds);
}

}  // namespace

hipError_t launch_grouped_ksplit(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                                 int format, int op_b) {
    constexpr int kGroupM = 8;
    const int tn = ceil_div(p.N, 64);
    const dim3 g((unsigned)(grouped_row_tiles(a.rows, a.groups, 64) * tn)), b(256);
    if (format == 0 && op_b) hipLaunchKernelGGL((grouped_ksplit_kernel<0, true>), g, b, 0, s, a, p, e, tn, kGroupM);
    else if (format == 0) hipLaunchKernelGGL((grouped_ksplit_kernel<0, false>), g, b, 0, s, a, p, e, tn, kGroupM);
    else if (op_b) hipLaunchKernelGGL((grouped_ksplit_kernel<1, true>), g, b, 0, s, a, p, e, tn, kGroupM);
    else hipLaunchKernelGGL((grouped_ksplit_kernel<1, false>), g, b, 0, s, a, p, e, tn, kGroupM);
    return hipGetLastError();
}

hipError_t launch_grouped_grad_ksplit(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                                      int format) {
    constexpr int kGroupM = 8;
    const int tm = ceil_div(p.M, 64), tn = ceil_div(p.N, 64);
    const dim3 g((unsigned)(tm * tn * a.groups)), b(256);
    if (format == 0) hipLaunchKernelGGL((grouped_grad_ksplit_kernel<0>), g, b, 0, s, a, p, e, tm, tn, kGroupM);
    else hipLaunchKernelGGL((grouped_grad_ksplit_kernel<1>), g, b, 0, s, a, p, e, tm, tn, kGroupM);
    return hipGetLastError();
}

}  // namespace gemmf32
