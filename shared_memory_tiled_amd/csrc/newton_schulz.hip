// newton_schulz.hip -- orthogonalisation of a matrix by Newton-Schulz
// products, as the Muon optimiser applies it to a weight's update.
//
//   X_0 = G / (|G|_F + eps)
//   A = X X^T,  B = b A + c A^2,  X <- a X + B X        (rows <= cols)
//   A = X^T X,  B = b A + c A^2,  X <- a X + X B        (rows > cols)
//
// Each step applies the odd polynomial a s + b s^3 + c s^5 to every singular
// value s of X and keeps the singular vectors.
#include "epilogue.h"

namespace gemmf32 {

namespace {

constexpr int kThreads = 256;
constexpr int kNormBlocks = 256;

// Partial sums of squares in binary64 (no overflow or underflow for any
// binary32 input), one per block and matrix.
template <int TYPE>
__global__ __launch_bounds__(kThreads)
void square_sum_kernel(NewtonSchulzArgs a, double* partials) {
    __shared__ double slots[kThreads];
    const int64_t base = (int64_t)blockIdx.y * a.stride_g;
    double s = 0.0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x)
        for (int c = threadIdx.x; c < a.cols; c += kThreads) {
            float v[1];
            load_values<TYPE>(a.G, base + r * a.ldg + c, 1, v);
            s += (double)v[0] * v[0];
        }
    slots[threadIdx.x] = s;
    for (int h = kThreads / 2; h > 0; h >>= 1) {
        __syncthreads();
        if ((int)threadIdx.x < h) slots[threadIdx.x] += slots[threadIdx.x + h];
    }
    if (threadIdx.x == 0) partials[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = slots[0];
}

template <int TYPE>
__global__ __launch_bounds__(kThreads)
void scale_kernel(NewtonSchulzArgs a, int64_t z, const double* partials, float* x) {
    double s = 0.0;
    for (int i = 0; i < kNormBlocks; ++i) s += partials[i];
    const float scale = (float)(1.0 / (sqrt(s) + (double)a.eps));
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.cols) return;
    float v[1];
    load_values<TYPE>(a.G, z * a.stride_g + (int64_t)blockIdx.y * a.ldg + c, 1, v);
    x[(int64_t)blockIdx.y * a.cols + c] = v[0] * scale;
}

// out = s u + t v over n values.
__global__ __launch_bounds__(kThreads)
void combine_kernel(int64_t n, float s, const float* u, float t, const float* v, float* out) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i < n) out[i] = s * u[i] + t * v[i];
}

__global__ __launch_bounds__(kThreads)
void write_kernel(NewtonSchulzArgs a, int64_t z, const float* x) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.cols) return;
    float v[1] = {x[(int64_t)blockIdx.y * a.cols + c]};
    store_values(a.type, a.out, z * a.stride_o + (int64_t)blockIdx.y * a.ldo + c, 1, v);
}

hipError_t product(int op_a, int op_b, int M, int N, int K, const float* A, int64_t lda, const float* B, int64_t ldb,
                   float* C, hipStream_t s) {
    const GemmArgs p{M, N, K, A, lda, B, ldb, C, N};
    return launch_mfma(p, s, mfma_pick_config(M, N, K), op_a, op_b);
}

}  // namespace

// |p(s)| on [0, bound], p(s) = a s + b s^3 + c s^5, is largest at the end or
// where p'(s) = a + 3 b s^2 + 5 c s^4 = 0; 1 % is added for the products'
// rounding.
bool newton_schulz_bounds(int steps, double a, double b, double c, double* bounds) {
    auto p = [&](double s) { return fabs(s * (a + s * s * (b + s * s * c))); };
    double bound = 1.01;
    for (int k = 0; k <= steps; ++k) {
        bounds[k] = bound;
        if (!(bound <= 1099511627776.0)) return false;
        double next = p(bound);
        const double disc = 9.0 * b * b - 20.0 * a * c;
        double roots[2] = {-1.0, -1.0};                  // of s^2
        if (c != 0.0 && disc >= 0.0) {
            roots[0] = (-3.0 * b + sqrt(disc)) / (10.0 * c);
            roots[1] = (-3.0 * b - sqrt(disc)) / (10.0 * c);
        } else if (c == 0.0 && b != 0.0) {
            roots[0] = -a / (3.0 * b);
        }
        for (const double r : roots)
            if (r > 0.0 && r < bound * bound) next = fmax(next, p(sqrt(r)));
        bound = 1.01 * next;
    }
    return true;
}

int64_t newton_schulz_workspace(const NewtonSchulzArgs& a) {
    const int64_t m = a.rows < a.cols ? a.rows : a.cols;
    return 8 * kNormBlocks * a.batch + 4 * (2 * (int64_t)a.rows * a.cols + 2 * m * m);
}

hipError_t launch_newton_schulz(const NewtonSchulzArgs& a, void* workspace, hipStream_t s) {
    double* const partials = static_cast<double*>(workspace);
    float* const x = reinterpret_cast<float*>(partials + kNormBlocks * a.batch);
    const int64_t mn = (int64_t)a.rows * a.cols;
    const int m = a.rows < a.cols ? a.rows : a.cols, n = a.rows < a.cols ? a.cols : a.rows;
    const bool wide = a.rows <= a.cols;
    float* const y = x + mn;
    float* const A = y + mn;
    float* const B = A + (int64_t)m * m;
    if (a.batch > 65535 || a.rows > 65535) return hipErrorInvalidValue;
    const dim3 ngrid(kNormBlocks, (unsigned)a.batch);
    if (a.type == 0) hipLaunchKernelGGL(square_sum_kernel<0>, ngrid, dim3(kThreads), 0, s, a, partials);
    else if (a.type == 1) hipLaunchKernelGGL(square_sum_kernel<1>, ngrid, dim3(kThreads), 0, s, a, partials);
    else hipLaunchKernelGGL(square_sum_kernel<2>, ngrid, dim3(kThreads), 0, s, a, partials);
    hipError_t e = hipGetLastError();
    const dim3 rgrid(ceil_div(a.cols, kThreads), a.rows);
    auto blocks = [](int64_t n_) { return dim3((unsigned)((n_ + kThreads - 1) / kThreads)); };
    for (int64_t z = 0; z < a.batch && e == hipSuccess; ++z) {
        const double* pz = partials + kNormBlocks * z;
        if (a.type == 0) hipLaunchKernelGGL(scale_kernel<0>, rgrid, dim3(kThreads), 0, s, a, z, pz, x);
        else if (a.type == 1) hipLaunchKernelGGL(scale_kernel<1>, rgrid, dim3(kThreads), 0, s, a, z, pz, x);
        else hipLaunchKernelGGL(scale_kernel<2>, rgrid, dim3(kThreads), 0, s, a, z, pz, x);
        e = hipGetLastError();
        const int ld = a.cols;
        for (int k = 0; k < a.steps && e == hipSuccess; ++k) {
            e = wide ? product(0, 1, m, m, n, x, ld, x, ld, A, s) : product(1, 0, m, m, n, x, ld, x, ld, A, s);
            if (e == hipSuccess) e = product(0, 0, m, m, m, A, m, A, m, B, s);
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL(combine_kernel, blocks((int64_t)m * m), dim3(kThreads), 0, s, (int64_t)m * m, a.b, A,
                               a.c, B, B);
            e = hipGetLastError();
            if (e == hipSuccess)
                e = wide ? product(0, 0, m, n, m, B, m, x, ld, y, s) : product(0, 0, n, m, m, x, ld, B, m, y, s);
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL(combine_kernel, blocks(mn), dim3(kThreads), 0, s, mn, a.a, x, 1.0f, y, x);
            e = hipGetLastError();
        }
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(write_kernel, rgrid, dim3(kThreads), 0, s, a, z, x);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace gemmf32
