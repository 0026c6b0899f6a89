// newton_schulz.hip -- orthogonalisation of a matrix by Newton-Schulz
// products, as the Muon optimiser applies it to a weight's update.
//
//   X_0 = G / (|G|_F + eps)
//   A = X X^T,  B = b A + c A^2,  X <- a X + B X        (rows <= cols)
//   A = X^T X,  B = b A + c A^2,  X <- a X + X B        (rows > cols)
//
// Each step applies the odd polynomial a s + b s^3 + c s^5 to every singular
// value s of X and keeps the singular vectors.
//
// Three products per step, on binary16 matrix instructions with binary32
// sums.  Every matrix is kept as two binary16 planes (newton_schulz_product.h;
// 22 bits).  Binary32 and binary16 results take the products of both planes
// (three matrix instructions for one: the product of the low planes, 2^-22 of
// the whole, is left out), whose error is below a binary32 product's at a
// third of the 16-bit rate instead of a sixteenth.  Bfloat16 results take the
// product of the high planes alone, X itself and the diagonals of A and B
// still in 22 and 24 bits: measured against binary64 their error, 5e-4 to
// 7e-4 of an entry's root mean square, is a third of the result's own
// rounding (1.7e-3), where products of bfloat16 factors give 1.4e-2 and more
// (matrices of at most 64 x 64 take both planes too, see the launcher).
// Scales are powers of two from bounds on the singular values, so no plane
// overflows; one scale serves a matrix.  The 22 bits hold for entries above
// 2^-16 of the norm; below, the low plane runs out of binary16's exponents, and
// half its last step, 2^-25 / 2^14 = 2^-39 of the norm, is what an entry is off
// by and below which it is 0.  Rows or columns so much smaller than the rest are
// not resolved (at 1e-6 of the largest row their error is 1.4e-4, at 1e-9 0.13 of
// them).  A scale per row and column would have to be undone in the products'
// inner sums, that is, in a second copy of X's planes written by every step.
#include "epilogue.h"
#include "newton_schulz_product.h"

namespace gemmf32 {

namespace {

constexpr int kThreads = 256;
constexpr int kNormBlocks = 256;

// The sum of squares in binary64 (no overflow or underflow for any binary32
// input).  Block b of matrix blockIdx.y takes runs of 8 columns in turn, four
// loads in flight (4096^2 bf16: 9.4 us, a row per block and turn 18.3).
template <int TYPE>
__global__ __launch_bounds__(kThreads)
void ns_square_sum_kernel(NewtonSchulzArgs a, double* partials) {
    __shared__ double slots[kThreads];
    const int64_t base = (int64_t)blockIdx.y * a.stride_g;
    const unsigned chunks = (unsigned)(a.cols + 7) / 8, total = chunks * (unsigned)a.rows;   // below 2^28
    constexpr unsigned STEP = kNormBlocks * kThreads;
    double s = 0.0;
    auto add = [&](const float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s += (double)v[e] * v[e];
    };
    unsigned i = blockIdx.x * kThreads + threadIdx.x;
    if (a.cols % 8 == 0) {                               // no run in part: loads without a branch
        for (; i + 3 * STEP < total; i += 4 * STEP) {
            float v[4][8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const unsigned r = (i + u * STEP) / chunks, c = 8 * (i + u * STEP - r * chunks);
                load_values<TYPE>(a.G, base + (int64_t)r * a.ldg + c, 8, v[u]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) add(v[u]);
        }
    }
    for (; i < total; i += STEP) {
        const unsigned r = i / chunks, c = 8 * (i - r * chunks);
        float v[8];
        load_values<TYPE>(a.G, base + (int64_t)r * a.ldg + c, a.cols - (int)c, v);
        add(v);
    }
    slots[threadIdx.x] = s;
    for (int h = kThreads / 2; h > 0; h >>= 1) {
        __syncthreads();
        if ((int)threadIdx.x < h) slots[threadIdx.x] += slots[threadIdx.x + h];
    }
    if (threadIdx.x == 0) partials[(int64_t)blockIdx.y * kNormBlocks + blockIdx.x] = slots[0];
}

// X_0's planes, padding included.  A norm that is no number or infinite
// makes every entry NaN.
template <int TYPE>
__global__ __launch_bounds__(kThreads)
void ns_split_kernel(NewtonSchulzArgs a, const double* partials, float x_scale, uint16_t* x, int rp, int cp,
                     int64_t stride) {
    __shared__ double slots[kThreads];
    slots[threadIdx.x] = partials[(int64_t)blockIdx.y * kNormBlocks + threadIdx.x];
    static_assert(kThreads == kNormBlocks, "one partial per thread");
    for (int h = kThreads / 2; h > 0; h >>= 1) {
        __syncthreads();
        if ((int)threadIdx.x < h) slots[threadIdx.x] += slots[threadIdx.x + h];
    }
    __syncthreads();
    const double norm = sqrt(slots[0]);
    const double scale = __builtin_isfinite(norm) ? (double)x_scale / (norm + (double)a.eps) : __builtin_nan("");
    const int64_t base = (int64_t)blockIdx.y * a.stride_g;
    const int chunks = cp / 8;
    const int64_t total = (int64_t)rp * chunks;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int r = (int)(i / chunks), c = 8 * (int)(i % chunks);
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < a.rows && c < a.cols) {
            load_values<TYPE>(a.G, base + (int64_t)r * a.ldg + c, a.cols - c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = c + e < a.cols ? (float)(v[e] * scale) : 0.0f;
        }
        store_planes<8, true>(x + (int64_t)blockIdx.y * stride, plane_index(r, cp, c), (int64_t)rp * cp, v);
    }
}

// No step: the planes' values into the result.
__global__ __launch_bounds__(kThreads)
void ns_write_kernel(NewtonSchulzArgs a, float unscale, const uint16_t* x, int rp, int cp, int64_t stride) {
    const int c = 8 * (blockIdx.x * kThreads + threadIdx.x);
    if (c >= a.cols) return;
    const int64_t z = blockIdx.z;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        float v[8];
        PlaneRun<8, true> run;
        run.load(x + z * stride, plane_index((int)r, cp, c), (int64_t)rp * cp);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = run.value(e) * unscale;
        store_values(a.type, a.out, z * a.stride_o + r * a.ldo + c, a.cols - c, v);
    }
}

// Workspace: partial norms, X's planes twice, S's and T's planes, d and e; then
// room for a large tile's rows past a matrix's last, which the product kernels
// copy and do not use (a copy's scalar offset, here the second plane's, is no
// part of its range check).
struct Layout {
    int rp, cp, mp;
    int64_t x_stride, s_stride;               // elements per matrix
    int64_t x0, x1, s, t, d, e, bytes;        // byte offsets
};
int pad64(int n) { return (n + 63) / 64 * 64; }
Layout layout(const NewtonSchulzArgs& a) {
    Layout l;
    l.rp = pad64(a.rows);
    l.cp = pad64(a.cols);
    l.mp = l.rp < l.cp ? l.rp : l.cp;
    l.x_stride = 2 * (int64_t)l.rp * l.cp;
    l.s_stride = 2 * (int64_t)l.mp * l.mp;
    l.x0 = 8 * (int64_t)kNormBlocks * a.batch;
    l.x1 = l.x0 + 2 * l.x_stride * a.batch;
    l.s = l.x1 + 2 * l.x_stride * a.batch;
    l.t = l.s + 2 * l.s_stride * a.batch;
    l.d = l.t + 2 * l.s_stride * a.batch;
    l.e = l.d + 4 * (int64_t)l.mp * a.batch;
    l.bytes = l.e + 4 * (int64_t)l.mp * a.batch + 2 * 256 * (int64_t)(l.rp > l.cp ? l.rp : l.cp);
    return l;
}

// The largest power of two that keeps values up to `bound` at most 2^15.
float plane_scale(double bound) { return (float)ldexp(1.0, 15 - (int)ceil(log2(fmax(bound, 1e-30)))); }

// The tiles a product runs on: those of the smallest estimated time, in us
// from the following measurements (MI355X, each kernel alone).
//   A round of 256 blocks takes the K loop, `slow` per 64-deep phase once all
//   CUs are busy (the clock drops, and the copies of the small tiles share
//   the L2; `fast` up to half of them), and `fixed` for start and epilogue by
//   stage.  4096^2, one term: Gram 84 / 67 / 81 / 124 us on 256 / 192 / 160 /
//   128 tiles (136, 253, 351 and 528 of them), update 114 / 141 / 176 / 207;
//   2048^2: update 53 / 38 / 34 / 31.
//   64 tiles: 3.3 + 0.0037 K per round (1024^2: Gram 6.7 against 15.3 us on
//   128 tiles; 4096^2 302 against 67).
int pick_tile(const NsProduct& p) {
    static const struct { int tile; double fast, slow, fixed[3]; } kTiles[] = {
        {256, 1.03, 1.50, {14.0, 23.0, 18.0}}, {192, 0.72, 0.90, {9.2, 14.0, 11.4}},
        {160, 0.62, 0.75, {7.3, 10.6, 8.7}}, {128, 0.37, 0.52, {9.7, 13.7, 12.5}}};
    const double k = (double)p.K * p.terms;
    const int64_t t64 = (int64_t)(p.M / 64) * (p.N / 64) * p.batch;
    int best = 64;
    double best_time = (double)((t64 + 255) / 256) * (3.3 + 0.0037 * k);
    const int stage = p.stage < kUpdate ? p.stage : kUpdate;
    for (const auto& w : kTiles) {
        const int64_t tm = ceil_div(p.M, w.tile), tn = ceil_div(p.N, w.tile);
        const int64_t tiles = (stage < kUpdate ? tm * (tm + 1) / 2 : tm * tn) * p.batch;
        const double busy = fmin(1.0, fmax(0.0, (double)tiles / 128.0 - 1.0));
        const double phase = w.fast + (w.slow - w.fast) * busy;
        const double time = (double)((tiles + 255) / 256) * (phase * k / 64.0 + w.fixed[stage]);
        if (time < best_time) {
            best_time = time;
            best = w.tile;
        }
    }
    return best;
}

hipError_t launch_product(const NsProduct& p, int op_a, hipStream_t s) {
    const int tile = pick_tile(p);
    if (tile == 64) return launch_ns_ksplit(p, op_a, s);
    if (tile == 128) return launch_ns_ksplit128(p, op_a, s);
    return launch_ns_wide(p, tile, op_a, s);
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
    // both planes of a matrix, padded to 64 and with a tile's overhang, within
    // 2^31 bytes; refused before anything is padded in 32 bits
    auto span = [](int n) { return ((int64_t)n + 63) / 64 * 64 + 256; };
    const int64_t rows = span(a.rows), cols = span(a.cols);      // below 2^32
    if (rows > ((1ll << 29) - 1) / cols || a.batch > 65535) return -1;   // 4 rows cols >= 2^31
    return layout(a).bytes;
}

hipError_t launch_newton_schulz(const NewtonSchulzArgs& a, void* workspace, hipStream_t s) {
    const Layout l = layout(a);
    char* const ws = static_cast<char*>(workspace);
    double* const partials = reinterpret_cast<double*>(ws);
    uint16_t* x = reinterpret_cast<uint16_t*>(ws + l.x0);
    uint16_t* x_next = reinterpret_cast<uint16_t*>(ws + l.x1);
    uint16_t* const S = reinterpret_cast<uint16_t*>(ws + l.s);
    uint16_t* const T = reinterpret_cast<uint16_t*>(ws + l.t);
    float* const d = reinterpret_cast<float*>(ws + l.d);
    float* const e = reinterpret_cast<float*>(ws + l.e);
    const unsigned batch = (unsigned)a.batch;
    const dim3 block(kThreads), ngrid(kNormBlocks, batch);
    const int64_t chunks = (int64_t)l.rp * l.cp / 8 / kThreads;          // cp is a multiple of 64
    const dim3 sgrid((unsigned)(chunks < 1 ? 1 : chunks > 2048 ? 2048 : chunks), batch);
    float sx = plane_scale(a.bounds[0]);
    if (a.type == 0) {
        hipLaunchKernelGGL(ns_square_sum_kernel<0>, ngrid, block, 0, s, a, partials);
        hipLaunchKernelGGL(ns_split_kernel<0>, sgrid, block, 0, s, a, partials, sx, x, l.rp, l.cp, l.x_stride);
    } else if (a.type == 1) {
        hipLaunchKernelGGL(ns_square_sum_kernel<1>, ngrid, block, 0, s, a, partials);
        hipLaunchKernelGGL(ns_split_kernel<1>, sgrid, block, 0, s, a, partials, sx, x, l.rp, l.cp, l.x_stride);
    } else {
        hipLaunchKernelGGL(ns_square_sum_kernel<2>, ngrid, block, 0, s, a, partials);
        hipLaunchKernelGGL(ns_split_kernel<2>, sgrid, block, 0, s, a, partials, sx, x, l.rp, l.cp, l.x_stride);
    }
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (a.steps == 0) {
        hipLaunchKernelGGL(ns_write_kernel, dim3(ceil_div(a.cols, 8 * kThreads), a.rows < 1024 ? a.rows : 1024, batch),
                           block, 0, s, a, 1.0f / sx, x, l.rp, l.cp, l.x_stride);
        return hipGetLastError();
    }
    const bool wide = a.rows <= a.cols;
    const int64_t x_plane = l.x_stride / 2, s_plane = l.s_stride / 2;
    // Matrices of one 64 x 64 tile have too few entries for the 11-bit factors'
    // errors to average out where singular values lie close together: of 4096
    // random 2 x 2 matrices the worst was 2.3e-2 of its root mean square off with
    // one term, 3.2e-3 (the result's rounding) with three; 8 x 8 4.8e-3 and 2.2e-3.
    // 64 x 64 takes 68 us in a graph for 59 with three.  From 80 x 80 on, and of long matrices,
    // the worst stays within 2.0e-3.
    const bool one_tile = l.rp == 64 && l.cp == 64;
    const int terms = a.type == 0 && !one_tile ? 1 : 3;
    for (int k = 0; k < a.steps; ++k) {
        const double bx = a.bounds[k], ba = bx * bx, bt = (fabs((double)a.b) + fabs((double)a.c) * ba) * ba * 1.01;
        const float ss = plane_scale(ba), st = plane_scale(bt);
        const float sx_next = plane_scale(a.bounds[k + 1]);
        NsProduct g{};
        g.batch = (int)a.batch;
        g.terms = terms;
        g.a = a.a;
        g.b = a.b;
        g.c = a.c;
        g.diag_n = l.mp;
        g.rows = a.rows;
        g.cols = a.cols;
        // S, d
        g.stage = kGram;
        g.M = g.N = l.mp;
        g.K = wide ? l.cp : l.rp;
        g.A = g.B = x;
        g.lda = g.ldb = l.cp;
        g.plane_a = g.plane_b = x_plane;
        g.stride_a = g.stride_b = l.x_stride;
        g.unscale = 1.0f / sx / sx;
        g.diag_out = d;
        g.out = S;
        g.ldo = l.mp;
        g.plane_o = s_plane;
        g.stride_o = l.s_stride;
        g.out_scale = ss;
        if ((err = launch_product(g, wide ? 0 : 1, s)) != hipSuccess) return err;
        // T, e
        g.stage = kPoly;
        g.K = l.mp;
        g.A = g.B = S;
        g.lda = g.ldb = l.mp;
        g.plane_a = g.plane_b = s_plane;
        g.stride_a = g.stride_b = l.s_stride;
        g.unscale = 1.0f / ss / ss;
        g.in = S;
        g.ldi = l.mp;
        g.plane_i = s_plane;
        g.stride_i = l.s_stride;
        g.in_unscale = 1.0f / ss;
        g.diag_in = d;
        g.diag_out = e;
        g.out = T;
        g.out_scale = st;
        if ((err = launch_product(g, 0, s)) != hipSuccess) return err;
        // X
        g.stage = wide ? kUpdate : kUpdateColumns;
        g.M = l.rp;
        g.N = l.cp;
        g.K = l.mp;
        if (wide) {
            g.B = x;
            g.ldb = l.cp;
            g.plane_b = x_plane;
            g.stride_b = l.x_stride;
            g.A = T;
        } else {
            g.A = x;
            g.lda = l.cp;
            g.plane_a = x_plane;
            g.stride_a = l.x_stride;
            g.B = T;
        }
        g.unscale = 1.0f / st / sx;
        g.in = x;
        g.ldi = l.cp;
        g.plane_i = x_plane;
        g.stride_i = l.x_stride;
        g.in_unscale = 1.0f / sx;
        g.diag_in = e;
        g.diag_out = nullptr;
        g.out = x_next;
        g.ldo = l.cp;
        g.plane_o = x_plane;
        g.stride_o = l.x_stride;
        g.out_scale = sx_next;
        if (k == a.steps - 1) {
            g.final_out = a.out;
            g.final_type = a.type;
            g.final_ld = a.ldo;
            g.final_stride = a.stride_o;
        }
        if ((err = launch_product(g, 0, s)) != hipSuccess) return err;
        uint16_t* const swap = x;
        x = x_next;
        x_next = swap;
        sx = sx_next;
    }
    return hipSuccess;
}

}  // namespace gemmf32
