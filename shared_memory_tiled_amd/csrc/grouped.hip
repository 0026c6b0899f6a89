// grouped.hip -- the layer whose rows belong to groups (experts) with a weight
// each: the passes over a split K's planes, and the activation's gradient with the
// groups' bias gradients.
//
// For the rows i of group g: Z_i = X_i W_g + b_g, Y_i = act(Z_i); backward,
// dZ = dY act'(Z), dX_i = dZ_i W_g^T (the same product with the weight's other
// orientation), dW_g = X_g^T dZ_g, db_g = the sum of dZ's rows of g.  The products
// are in grouped_shared.hip, the choice of their tiles in grouped_plan.h.
#include "epilogue.h"
#include "grouped_kernels.h"
#include "grouped_plan.h"

namespace gemmf32 {

namespace {

// ------------------------------------------- passes over a split K's planes

// W values at `at` of each plane, added in order, four loads in flight.
template <int W>
__device__ __forceinline__ void add_planes(const float* planes, int count, int64_t plane, int64_t at, int valid, float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = 0.0f;
    for (int q = 0; q < count; q += 4) {
        float u[4][W];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (q + k < count) load_values<2>(planes + (q + k) * plane, at, valid, u[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (q + k < count) {
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] += u[k][i];
            }
    }
}

// The layer's epilogue over the planes' sums: 16 rows of one group x 128 columns
// to a block, a run of 4 columns of two rows to a thread.
constexpr int kPassRows = 16;
__global__ __launch_bounds__(256)
void grouped_pass_kernel(GroupedArgs a, EpilogueArgs e, int tiles_n, const float* planes, int count, int64_t plane) {
    const GroupRows r = locate_group_tile<kPassRows>(a, (int)blockIdx.x, tiles_n, 1);
    if (r.rows < 0) return;
    Gemm16Args p{};
    enter_group(a, r, &p, &e);
    const int col = 128 * r.tn + 4 * (threadIdx.x & 31);
    if (col >= e.N) return;
    float bias[4];
    load_bias(e, col, bias);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = kPassRows * r.tm + (threadIdx.x >> 5) + 8 * h;
        if (row >= e.M) return;
        EpilogueRun<4, false> run;
        run.load(e, row, col);
        float v[4];
        add_planes(planes, count, plane, (int64_t)(r.begin + row) * e.N + col, e.N - col, v);
        run.finish(e, row, col, bias, v);
    }
}

// The gradients of all groups: rows are groups x M, 8 of them x 128 columns to a
// block.
__global__ __launch_bounds__(256)
void grouped_grad_pass_kernel(EpilogueArgs e, int64_t stride_c, int64_t rows, const float* planes, int count, int64_t plane) {
    const int64_t i = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5);
    const int col = 128 * blockIdx.x + 4 * (threadIdx.x & 31);
    if (i >= rows || col >= e.N) return;
    float v[4];
    add_planes(planes, count, plane, i * e.N + col, e.N - col, v);
    const int64_t g = i / e.M;
    store_values(e.c_type, e.C, g * stride_c + (i - g * e.M) * e.ldc + col, e.N - col, v);
}

}  // namespace

int64_t grouped_workspace(const GroupedArgs& a, const Gemm16Args& p, int op_b) {
    return make_plan(a, p, op_b).bytes;
}

hipError_t launch_grouped(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format,
                          int op_b, void* workspace) {
    const Plan q = make_plan(a, p, op_b);
    if (q.splits == 1) return launch_grouped_shared(a, p, e, s, format, op_b, q.direct, q.bm, q.bn, q.k_share, 0);
    const int64_t plane = (int64_t)a.rows * p.N;
    EpilogueArgs sums{};
    sums.N = e.N;
    sums.c_type = 2;
    sums.C = workspace;
    sums.ldc = p.N;
    const hipError_t err = launch_grouped_shared(a, p, sums, s, format, op_b, q.direct, q.bm, q.bn, q.k_share, plane);
    if (err != hipSuccess) return err;
    const int tn = ceil_div(e.N, 128);
    hipLaunchKernelGGL(grouped_pass_kernel, dim3((unsigned)(grouped_row_tiles(a.rows, a.groups, kPassRows) * tn)), dim3(256),
                       0, s, a, e, tn, static_cast<const float*>(workspace), q.splits, plane);
    return hipGetLastError();
}

int64_t grouped_grad_workspace(const GroupedArgs& a, const Gemm16Args& p) {
    return make_grad_plan(a, p).bytes;
}

hipError_t launch_grouped_grad(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                               int format, void* workspace) {
    const Plan q = make_grad_plan(a, p);
    if (q.splits == 1) return launch_grouped_grad_shared(a, p, e, s, format, q.direct, q.bn, 1, 0);
    const int64_t plane = (int64_t)a.groups * p.M * p.N;
    GroupedArgs whole = a;
    whole.stride_b = (int64_t)p.M * p.N;
    EpilogueArgs sums{};
    sums.M = p.M;
    sums.N = p.N;
    sums.c_type = 2;
    sums.C = workspace;
    sums.ldc = p.N;
    const hipError_t err = launch_grouped_grad_shared(whole, p, sums, s, format, q.direct, q.bn, q.splits, plane);
    if (err != hipSuccess) return err;
    const int64_t rows = (int64_t)a.groups * p.M;
    hipLaunchKernelGGL(grouped_grad_pass_kernel, dim3(ceil_div(p.N, 128), (unsigned)((rows + 7) / 8)), dim3(256), 0, s, e,
                       a.stride_b, rows, static_cast<const float*>(workspace), q.splits, plane);
    return hipGetLastError();
}

// --------------------------------------------- the activation's gradient

namespace {

// Bound by memory: 8192 x 2048 bf16 over 16 groups 25 us alone (4 TB/s), 28 to 32
// within a backward pass, where what it writes stays in the caches for the
// products.  1000 x 500 over 6 groups, with the sums, 14 us: two launches of a
// row's latency each.
//
// dZ is stored in 16 bits, since the products that read it take 16-bit factors:
// against binary64 the pass's results are 1.41 times as far off as with an unrounded
// dZ (8192 x 2048 x 4096 bf16 2.3e-3 of the root mean square, 1.66e-3 of which is the
// results' own rounding; f16 2.9e-4 and 2.1e-4).  The groups' sums are of dZ before it.
//
// dZ = dY act'(Z) over tiles of kActRows rows of one group x 256 columns, a
// thread 8 columns of every eighth row; the tile's column sums, of dZ before
// its rounding, go to partials[tile][N].  One tile row per row tile of the
// groups; the last block of a column adds nothing: a second kernel adds each
// group's tiles in order.
constexpr int kActRows = 64, kActCols = 256;
__global__ __launch_bounds__(256)
void grouped_activation_kernel(GroupedArgs a, EpilogueArgs e, const uint16_t* dY, int64_t ld, int tiles_n, float* partials) {
    __shared__ float part[8][kActCols];
    const GroupRows r = locate_group_tile<kActRows>(a, (int)blockIdx.x, tiles_n, 1 << 20);
    if (r.rows < 0) return;
    const int c = 8 * (threadIdx.x & 31), w = threadIdx.x >> 5, col = r.tn * kActCols + c;
    const int first = r.tm * kActRows, last = min(first + kActRows, r.rows);
    float sums[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    // Four rows' loads in flight: one row after the other, a small layer's pass is
    // eight times the memory's latency (90 x 171 13 us).  A run across N is loaded
    // from further down in its row and moved; rows shorter than a run go one by
    // one.
    const bool z = e.act != kActNone;
    const uint16_t* const pre = static_cast<const uint16_t*>(e.preact);
    if (col < e.N) {
        const int from = max(min(col, e.N - 8), 0), by = col - from;
        auto load = [&](const uint16_t* row) __attribute__((always_inline)) -> u32x4 {
            u32x4 v = {0, 0, 0, 0};
            if (e.N >= 8) __builtin_memcpy(&v, row + from, 16);
            else
                for (int k = 0; k < e.N; ++k) v[k / 2] |= (unsigned)row[k] << (16 * (k % 2));
            return v;
        };
        auto values = [&](u32x4 v, float (&f)[8]) __attribute__((always_inline)) {
            RawRun<8> run;
            v = move_down(v, by);
            __builtin_memcpy(run.w, &v, 16);
            run.values(e.z_type, f);
        };
        for (int i = first + w; i < last; i += 32) {
            u32x4 yr[4], zr[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {                  // past the last row: that one again
                const int64_t row = r.begin + min(i + 8 * u, last - 1);
                yr[u] = load(dY + row * ld);
                if (z) zr[u] = load(pre + row * e.ldz);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + 8 * u < last) {
                    const int64_t row = r.begin + i + 8 * u;
                    float v[8], zv[8];
                    values(yr[u], v);
                    if (z) {
                        values(zr[u], zv);
                        times_derivative(e.act, zv, v);
                    }
                    if (e.C != nullptr) store_values(e.c_type, e.C, row * e.ldc + col, e.N - col, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) sums[k] += v[k];
                }
        }
    }
    if (partials == nullptr) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) part[w][c + k] = sums[k];
    __syncthreads();
    const int at = threadIdx.x, out = r.tn * kActCols + at;
    if (out >= e.N) return;
    float s = part[0][at];
#pragma unroll
    for (int k = 1; k < 8; ++k) s += part[k][at];
    // The row tile's number over all groups: the tiles of the groups before
    // end where this group's begin, at most one more per group than whole ones.
    partials[((int64_t)r.begin / kActRows + r.group + r.tm) * e.N + out] = s;
}

// db[g][n] = the sum of group g's tiles, in order; a block per 64 columns and
// group, four tiles at a time.
__global__ __launch_bounds__(256)
void grouped_sum_kernel(GroupedArgs a, int N, const float* partials, float* out) {
    __shared__ float part[4][64];
    int begin, end;
    const int g = blockIdx.y;
    group_range(a, g, &begin, &end);
    const int col = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
    const int tiles = (end - begin + kActRows - 1) / kActRows;
    const float* const q = partials + ((int64_t)begin / kActRows + g) * N;
    float s = 0.f;
    if (col < N)
        for (int i = w; i < tiles; i += 32) {              // eight loads in flight, added in order
            float u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = i + 4 * k < tiles ? q[(int64_t)(i + 4 * k) * N + col] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += u[k];
        }
    part[w][threadIdx.x & 63] = s;
    __syncthreads();
    if (w == 0 && col < N)
        out[(int64_t)g * N + col] = ((part[0][threadIdx.x] + part[1][threadIdx.x]) + part[2][threadIdx.x]) + part[3][threadIdx.x];
}

}  // namespace

// Tile t of group g is partials row begin_g / kActRows + g + t.  Rows of
// different groups do not meet: begin / 64 + tiles <= end / 64 + 1 for any
// range, so a group's last row is below the next group's first.
int64_t grouped_activation_workspace(int64_t rows, int64_t groups, int64_t N) {
    return 4 * (rows / kActRows + groups + 1) * N;
}

hipError_t launch_grouped_activation(const GroupedArgs& a, const EpilogueArgs& e, const uint16_t* dY, int64_t ld,
                                     float* partials, hipStream_t s) {
    const int tn = ceil_div(e.N, kActCols);
    const int64_t blocks = grouped_row_tiles(a.rows, a.groups, kActRows) * tn;
    if (blocks > 0x7FFFFFFFll / 256 || a.groups > 65535) return hipErrorInvalidValue;
    float* const part = e.bias_grad != nullptr ? partials : nullptr;
    if (blocks > 0) {
        hipLaunchKernelGGL(grouped_activation_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, e, dY, ld, tn, part);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (part == nullptr) return hipSuccess;
    hipLaunchKernelGGL(grouped_sum_kernel, dim3(ceil_div(e.N, 64), (unsigned)a.groups), dim3(256), 0, s, a, e.N, part,
                       e.bias_grad);
    return hipGetLastError();
}

}  // namespace gemmf32
