// grouped.hip -- the layer whose rows belong to groups (experts) with a weight
// each: choice of tile, the passes over a split K's planes, and the activation's
// gradient with the groups' bias gradients.
//
// For the rows i of group g: Z_i = X_i W_g + b_g, Y_i = act(Z_i); backward,
// dZ = dY act'(Z), dX_i = dZ_i W_g^T (the same product with the weight's other
// orientation), dW_g = X_g^T dZ_g, db_g = the sum of dZ's rows of g.  The products
// are in grouped_shared.hip.
#include "epilogue.h"
#include "grouped_kernels.h"

#include <math.h>

namespace gemmf32 {

namespace {

// ------------------------------------------------------- choice of kernel

// A factor of `rows` rows whose copies' 32-bit offsets hold, a tile's
// overhang included.
bool offsets_hold(int64_t rows, int64_t ld) { return ld < (1ll << 30) / (rows + 256); }
bool even_base(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Whether the operands can be copied straight into LDS.
bool direct_fits(const GroupedArgs& a, const Gemm16Args& p, int op_b) {
    return p.K > 0 && p.K % 2 == 0 && p.lda % 2 == 0 && p.ldb % 2 == 0 && a.stride_b % 2 == 0 && (op_b || p.N % 2 == 0) &&
           even_base(p.A) && even_base(p.B) && offsets_hold(256, p.lda) && offsets_hold(op_b ? p.N : p.K, p.ldb);
}
bool direct_grad_fits(const GroupedArgs& a, const Gemm16Args& p) {
    return p.lda % 2 == 0 && p.ldb % 2 == 0 && p.M % 2 == 0 && p.N % 2 == 0 && even_base(p.A) && even_base(p.B) &&
           offsets_hold(a.rows, p.lda) && offsets_hold(a.rows, p.ldb);
}

// Groups that have a row, if every row chooses one with the same chance.
double used_groups(int groups, int rows) { return groups * (1.0 - pow(1.0 - 1.0 / groups, rows)); }

// Row tiles that the groups make on average: each group leaves half a tile.
double expected_row_tiles(int groups, int rows, int tile) {
    if (groups == 1) return ceil_div(rows, tile);
    const double used = used_groups(groups, rows);
    return used * fmax(1.0, rows / used / tile + 0.5);
}

// Estimated time of `tiles` tiles of `phases` steps of 32 k, in us.  A block
// alone on a CU takes `alone` per phase, which is the memory's latency over the
// stages in flight; with `slots` of them on the chip (two or three to a CU) a
// round of them takes `full` per phase; and `fixed` for start and epilogue.  How
// many rounds the groups' rows make is not known here: past one, half a round
// more for the last.  (4096^3 in one group: 121 us on 128 x 256 tiles, 157 on 128
// x 128, 157 on 64 x 256, 185 on 64 x 128; 1024 x 1024 x 1024 in 16 groups: 28 /
// 19 / 19 / 15.)
struct Shape {
    int bm, bn, slots;
    double alone, full, fixed;
};
constexpr Shape kShapes[] = {
    {128, 256, 512, 0.45, 0.84, 13.5}, {128, 128, 768, 0.43, 0.875, 5.1}, {64, 256, 512, 0.45, 0.575, 5.0},
    {64, 128, 768, 0.305, 0.50, 5.0}};
double tiles_time(const Shape& c, double tiles, double phases) {
    if (tiles > c.slots) return (tiles / c.slots + 0.5) * (c.full * phases + c.fixed);
    const double busy = fmax(0.0, (tiles - 256.0) / (c.slots - 256.0));
    return (c.alone + (c.full - c.alone) * busy) * phases + c.fixed;
}

// The pass over `splits` planes of `values`, from 4 us, at 3 TB/s.
double pass_time(int splits, double values) { return 4.0 + 4.0 * splits * values / 3e6; }

struct Plan {
    bool direct;
    int bm, bn;
    int splits, k_share;               // blocks along K; k of each
    int64_t bytes;                     // of planes, if split
};

Plan make_plan(const GroupedArgs& a, const Gemm16Args& p, int op_b) {
    Plan q{};
    q.splits = 1;
    q.k_share = p.K;
    q.direct = direct_fits(a, p, op_b);
    if (p.K == 0) {                    // the epilogue alone
        q.bm = 64;
        q.bn = 128;
        q.k_share = 1;
        return q;
    }
    const int phases = ceil_div(p.K, 32);
    double least = 1e30;
    for (const Shape& c : kShapes) {
        if (!q.direct && c.bn != 128) continue;
        const double tiles = expected_row_tiles(a.groups, a.rows, c.bm) * ceil_div(p.N, c.bn);
        for (int splits = 1; splits <= 16 && (splits == 1 || (tiles * splits <= c.slots && phases >= 8 * splits)); splits *= 2) {
            const double t = tiles_time(c, tiles * splits, (double)phases / splits) +
                             (splits > 1 ? pass_time(splits, (double)a.rows * p.N) : 0.0);
            if (t < least) {
                least = t;
                q.bm = c.bm;
                q.bn = c.bn;
                q.k_share = splits > 1 ? 32 * ceil_div(phases, splits) : p.K;
                q.splits = ceil_div(p.K, q.k_share);
            }
        }
    }
    if (q.splits > 1) q.bytes = 4 * (int64_t)q.splits * a.rows * p.N;
    return q;
}

// The weights' gradient: 128 x 256 tiles for groups of 384 rows and more that make
// about one whole round of the 512 on the chip or two and more (16384 x 2048 x 4096
// over 2 groups 249 us against 294 on 128 x 128, 8192 x 2048 x 4096 over 16 147
// against 161), else 128 x 128, which store sooner (4096 x 1024 x 2048 over 64 63
// us against 70, 2000 x 1000 x 1000 over 4 15 against 20); few tiles with long
// groups split the rows.
Plan make_grad_plan(const GroupedArgs& a, const Gemm16Args& p) {
    Plan q{};
    q.splits = 1;
    q.direct = direct_grad_fits(a, p);
    q.bm = 128;
    const int64_t wide = (int64_t)a.groups * ceil_div(p.M, 128) * ceil_div(p.N, 256);
    const double rows = a.rows / used_groups(a.groups, a.rows > 0 ? a.rows : 1);
    q.bn = q.direct && rows >= 384 && ((wide >= 448 && wide <= 512) || wide >= 1024) ? 256 : 128;
    if (q.bn == 256) return q;
    const double tiles = (double)a.groups * ceil_div(p.M, 128) * ceil_div(p.N, 128);
    const double phases = ceil(rows / 32.0);
    double least = 1e30;
    for (int splits = 1; splits <= 32 && (splits == 1 || (tiles * splits <= 768 && phases >= 8 * splits)); splits *= 2) {
        const double t = tiles_time(kShapes[1], tiles * splits, phases / splits) +
                         (splits > 1 ? pass_time(splits, (double)a.groups * p.M * p.N) : 0.0);
        if (t < least) {
            least = t;
            q.splits = splits;
        }
    }
    if (q.splits > 1) q.bytes = 4 * (int64_t)q.splits * a.groups * p.M * p.N;
    return q;
}

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
