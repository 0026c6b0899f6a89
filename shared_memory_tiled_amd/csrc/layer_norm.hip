// layer_norm.hip -- layer norm over the rows of a matrix, forward and
// backward.
//
//   mean = <x>, rstd = 1 / sqrt(<(x - mean)^2> + eps), xhat = (x - mean) rstd
//   y  = xhat gamma + beta
//   g  = dy gamma;  dx = rstd (g - <g> - xhat <g xhat>) + residual_grad
//   dgamma = sum over rows of dy xhat;  dbeta = sum over rows of dy
//
// <.> is the mean over a row.  All statistics and sums are binary32; y and dx
// are rounded once.  The reductions are the block reductions of reduce.hip
// (wave shuffles, then LDS), one per row.
#include "epilogue.h"

namespace gemmf32 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float wave_total(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
// The block's sum of v in every thread (slots: one float per wave).
__device__ __forceinline__ float block_total(float v, float* slots) {
    v = wave_total(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    return (slots[0] + slots[1]) + (slots[2] + slots[3]);
}

template <int TYPE>
__global__ __launch_bounds__(kThreads)
void layer_norm_kernel(LayerNormArgs a) {
    __shared__ float slots[4];
    const int64_t row = blockIdx.x;
    float s = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        float v[1];
        load_values<TYPE>(a.x, row * a.ldx + c, 1, v);
        s += v[0];
    }
    const float mean = block_total(s, slots) / (float)a.cols;
    s = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        float v[1];
        load_values<TYPE>(a.x, row * a.ldx + c, 1, v);
        s += (v[0] - mean) * (v[0] - mean);
    }
    const float rstd = 1.0f / sqrtf(block_total(s, slots) / (float)a.cols + a.eps);
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        float v[1], g[1] = {1.f}, b[1] = {0.f};
        load_values<TYPE>(a.x, row * a.ldx + c, 1, v);
        if (a.gamma) load_values(a.param_type, a.gamma, c, 1, g);
        if (a.beta) load_values(a.param_type, a.beta, c, 1, b);
        v[0] = (v[0] - mean) * rstd * g[0] + b[0];
        store_values<TYPE>(a.y, row * a.ldy + c, 1, v);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

template <int TYPE>
__global__ __launch_bounds__(kThreads)
void layer_norm_backward_row_kernel(LayerNormArgs a) {
    __shared__ float slots[4];
    const int64_t row = blockIdx.x;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s0 = 0.f, s1 = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        float x[1], dy[1], g[1] = {1.f};
        load_values<TYPE>(a.x, row * a.ldx + c, 1, x);
        load_values<TYPE>(a.dy, row * a.lddy + c, 1, dy);
        if (a.gamma) load_values(a.param_type, a.gamma, c, 1, g);
        s0 += dy[0] * g[0];
        s1 += dy[0] * g[0] * ((x[0] - mean) * rstd);
    }
    const float m0 = block_total(s0, slots) / (float)a.cols, m1 = block_total(s1, slots) / (float)a.cols;
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        float x[1], dy[1], g[1] = {1.f}, r[1] = {0.f};
        load_values<TYPE>(a.x, row * a.ldx + c, 1, x);
        load_values<TYPE>(a.dy, row * a.lddy + c, 1, dy);
        if (a.gamma) load_values(a.param_type, a.gamma, c, 1, g);
        if (a.residual_grad) load_values<TYPE>(a.residual_grad, row * a.ldr + c, 1, r);
        const float xhat = (x[0] - mean) * rstd;
        r[0] += rstd * (dy[0] * g[0] - m0 - xhat * m1);
        store_values<TYPE>(a.dx, row * a.lddx + c, 1, r);
    }
}

// Column sums of rows blockIdx.y rows_per_block .. : dgamma's, then dbeta's
// partials, one row of a.cols floats per block row each.
template <int TYPE>
__global__ __launch_bounds__(kThreads)
void layer_norm_backward_column_kernel(LayerNormArgs a, int64_t rows_per_block, float* part_g, float* part_b) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.cols) return;
    const int64_t r0 = blockIdx.y * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < a.rows ? r0 + rows_per_block : a.rows;
    float sg = 0.f, sb = 0.f;
    for (int64_t row = r0; row < r1; ++row) {
        float x[1], dy[1];
        load_values<TYPE>(a.x, row * a.ldx + c, 1, x);
        load_values<TYPE>(a.dy, row * a.lddy + c, 1, dy);
        sg += dy[0] * ((x[0] - a.mean[row]) * a.rstd[row]);
        sb += dy[0];
    }
    part_g[(int64_t)blockIdx.y * a.cols + c] = sg;
    part_b[(int64_t)blockIdx.y * a.cols + c] = sb;
}

int64_t column_blocks(int64_t rows) { return rows < 256 ? (rows + 7) / 8 : 256; }

template <int TYPE>
hipError_t launch_backward(const LayerNormArgs& a, void* workspace, hipStream_t s) {
    // the column sums first: dx may be dy
    hipError_t e = hipSuccess;
    if (a.dgamma != nullptr || a.dbeta != nullptr) {
        const int64_t blocks = column_blocks(a.rows), per = (a.rows + blocks - 1) / blocks;
        float* const pg = static_cast<float*>(workspace);
        float* const pb = pg + blocks * a.cols;
        hipLaunchKernelGGL(layer_norm_backward_column_kernel<TYPE>,
                           dim3(ceil_div(a.cols, kThreads), (unsigned)blocks), dim3(kThreads), 0, s, a, per, pg, pb);
        e = hipGetLastError();
        if (e == hipSuccess && a.dgamma) e = launch_column_sums((int)blocks, a.cols, pg, a.dgamma, s);
        if (e == hipSuccess && a.dbeta) e = launch_column_sums((int)blocks, a.cols, pb, a.dbeta, s);
    }
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(layer_norm_backward_row_kernel<TYPE>, dim3((unsigned)a.rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.rows);
    if (a.type == 0) hipLaunchKernelGGL(layer_norm_kernel<0>, grid, dim3(kThreads), 0, s, a);
    else if (a.type == 1) hipLaunchKernelGGL(layer_norm_kernel<1>, grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(layer_norm_kernel<2>, grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

int64_t layer_norm_backward_workspace(int /*type*/, int64_t rows, int cols) { return 2 * 4 * column_blocks(rows) * cols; }

hipError_t launch_layer_norm_backward(const LayerNormArgs& a, void* workspace, hipStream_t s) {
    if (a.type == 0) return launch_backward<0>(a, workspace, s);
    if (a.type == 1) return launch_backward<1>(a, workspace, s);
    return launch_backward<2>(a, workspace, s);
}

}  // namespace gemmf32
