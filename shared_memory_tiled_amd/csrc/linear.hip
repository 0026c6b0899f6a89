// linear.hip -- the fully connected layer's product with its epilogue (bias,
// activation, residual; or, backward, the activation's derivative and the
// bias gradient): choice of kernel, and the passes around the products.
//
// Z = op(A) op(B) + bias, C = act(Z) + residual; backward, D = (op(A) op(B)
// + residual) act'(Z) with D's column sums.  The one-volume PMPP notes run
// the layer and its backward pass as matrix products (deep-learning chapter,
// "FC Layer = GEMM", "Backward"); what follows the product there is done
// here before the entry leaves the chip.
//
// epilogue_kernel is the pass over finished sums: it adds the planes of a
// product whose K was split over blocks (or reads a matrix of 16-bit
// gradients), applies the epilogue and leaves column sums of its block of
// rows, which column_sum_kernel adds in row order (deterministic).
#include "epilogue.h"

#include <limits.h>

namespace gemmf32 {

namespace {

// Column tile of 128 (32 threads of 4 columns), 8 rows at a time,
// `rows_per_block` rows per block.  IN: 0, 1 a matrix of 16-bit values of
// that format, 2 `planes` binary32 planes of plane_stride floats, added in
// order.
constexpr int kPassCols = 128;
template <int IN>
__global__ __launch_bounds__(256)
void epilogue_kernel(EpilogueArgs e, const void* in, int64_t ld, int planes, int64_t plane_stride,
                     int rows_per_block, float* partials) {
    const int tc = threadIdx.x % 32, tr = threadIdx.x / 32;
    const int col = blockIdx.x * kPassCols + 4 * tc;
    const int first = blockIdx.y * rows_per_block;
    const int last = min(e.M, first + rows_per_block);
    float sums[4] = {0.f, 0.f, 0.f, 0.f};
    if (col < e.N) {
        for (int row = first + tr; row < last; row += 8) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (IN == 2) {
                for (int s = 0; s < planes; ++s) {
                    float w[4];
                    load_values<2>(in, s * plane_stride + (int64_t)row * ld + col, e.N - col, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += w[i];
                }
            } else {
                load_values<IN>(in, (int64_t)row * ld + col, e.N - col, v);
            }
            finish_entries(e, row, col, v);
            if (e.gradient) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[i] += v[i];
            }
        }
    }
    if (partials == nullptr) return;                     // the same for every thread
    __shared__ float part[8][kPassCols];
#pragma unroll
    for (int i = 0; i < 4; ++i) part[tr][4 * tc + i] = sums[i];
    __syncthreads();
    const int c = blockIdx.x * kPassCols + threadIdx.x;
    if (threadIdx.x < kPassCols && c < e.N) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
        partials[(int64_t)blockIdx.y * e.N + c] = s;
    }
}

// out[c] = sum of partials[i][c], i < count, in a fixed order: 8 threads take
// every eighth partial of a column, their sums are added in thread order.
__global__ __launch_bounds__(256)
void column_sum_kernel(int count, int n, const float* partials, float* out) {
    __shared__ float part[8][32];
    const int tc = threadIdx.x % 32, tr = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + tc;
    float s = 0.f;
    if (c < n)
        for (int i = tr; i < count; i += 8) s += partials[(int64_t)i * n + c];
    part[tr][tc] = s;
    __syncthreads();
    if (tr == 0 && c < n) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += part[i][tc];
        out[c] = t;
    }
}

// Rows per block of the pass: enough blocks for the device's 256 CUs (eight
// each), then as many rows as that leaves, for fewer partial sums.
int pass_rows(int M, int N) {
    const int64_t cols = ceil_div(N, kPassCols);
    const int64_t rows = ((int64_t)M * cols + 2047) / 2048;
    return 8 * (int)((rows + 7) / 8 > 0 ? (rows + 7) / 8 : 1);
}

int64_t align256(int64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

hipError_t launch_column_sums(int count, int n, const float* partials, float* out, hipStream_t s) {
    hipLaunchKernelGGL(column_sum_kernel, dim3(ceil_div(n, 32)), dim3(256), 0, s, count, n, partials, out);
    return hipGetLastError();
}

// Bytes of partial column sums the pass over an M x N matrix leaves.
int64_t epilogue_pass_workspace(int M, int N) {
    return align256(4 * (int64_t)ceil_div(M, pass_rows(M, N)) * N);
}

hipError_t launch_epilogue_pass(const EpilogueArgs& e, int in_type, const void* in, int64_t ld, int planes,
                                int64_t plane_stride, float* partials, hipStream_t s) {
    const int rpb = pass_rows(e.M, e.N);
    const int64_t gy = ceil_div(e.M, rpb);
    if (gy > 65535) return hipErrorInvalidValue;
    const dim3 grid(ceil_div(e.N, kPassCols), (unsigned)gy);
    float* const part = e.bias_grad != nullptr ? partials : nullptr;
    if (in_type == 0)
        hipLaunchKernelGGL(epilogue_kernel<0>, grid, dim3(256), 0, s, e, in, ld, planes, plane_stride, rpb, part);
    else if (in_type == 1)
        hipLaunchKernelGGL(epilogue_kernel<1>, grid, dim3(256), 0, s, e, in, ld, planes, plane_stride, rpb, part);
    else
        hipLaunchKernelGGL(epilogue_kernel<2>, grid, dim3(256), 0, s, e, in, ld, planes, plane_stride, rpb, part);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || part == nullptr) return err;
    return launch_column_sums((int)gy, e.N, part, e.bias_grad, s);
}

int64_t linear_workspace(const Gemm16Args& p, const EpilogueArgs& e, int, int) {
    return align256(4 * (int64_t)p.M * p.N) + (e.bias_grad ? epilogue_pass_workspace(p.M, p.N) : 0);
}

hipError_t launch_linear(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a, int op_b,
                         void* workspace) {
    Gemm16Args q = p;
    q.C = static_cast<float*>(workspace);
    q.ldc = p.N;
    const hipError_t err = (op_a || op_b) ? launch_mixed_op(q, s, format, op_a, op_b)
                                          : launch_mixed(q, s, format, mixed_pick_config(q.M, q.N, q.K));
    if (err != hipSuccess) return err;
    float* const partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256(4 * (int64_t)p.M * p.N));
    return launch_epilogue_pass(e, 2, q.C, q.ldc, 1, 0, partials, s);
}

}  // namespace gemmf32
