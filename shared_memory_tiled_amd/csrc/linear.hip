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
// The product runs on the tiles of least estimated time (pick_tile, below),
// on the few-row kernel up to 64 rows, split by rows on 256 x 256 tiles and
// smaller ones for the rest, or, few tiles and a long K, with K split over
// blocks.  Factors those kernels do not take (an odd width, leading dimension
// or K, a base of 2-byte alignment) are first copied into the workspace with
// padded rows: that costs less than the product's element-wise kernels would
// (999 x 1001 x 1001: 15 us against 100).  What is left (factors of 2 GiB and
// more, K = 0) runs the library's product into a binary32 matrix in the
// workspace and the epilogue as a pass over it.
//
// epilogue_kernel is the pass over finished sums: it adds the planes of a
// product whose K was split over blocks (or reads a matrix of 16-bit
// gradients), applies the epilogue and leaves column sums of its block of
// rows, which column_sum_kernel adds in row order (deterministic).
#include "epilogue.h"
#include "linear_kernels.h"

#include <limits.h>
#include <math.h>

namespace gemmf32 {

namespace {

// Column tile of 128 (32 threads of 4 columns), 8 rows at a time,
// `rows_per_block` rows per block.  IN: 0, 1 a matrix of 16-bit values of
// that format, 2 `planes` binary32 planes of plane_stride floats, added in
// order, eight loads in flight.
constexpr int kPassCols = 128;
template <int IN, bool GRADIENT>
__global__ __launch_bounds__(256)
void epilogue_kernel(EpilogueArgs e, const void* in, int64_t ld, int planes, int64_t plane_stride,
                     int rows_per_block, float* partials) {
    const int tc = threadIdx.x % 32, tr = threadIdx.x / 32;
    const int col = blockIdx.x * kPassCols + 4 * tc;
    const int first = blockIdx.y * rows_per_block;
    const int rows = min(e.M - first, rows_per_block);       // first + rows_per_block may pass 2^31
    float sums[4] = {0.f, 0.f, 0.f, 0.f};
    if (col < e.N) {
        float bias[4];
        if constexpr (!GRADIENT) load_bias(e, col, bias);
        for (int r = tr; r < rows; r += 8) {
            const int row = first + r;
            EpilogueRun<4, GRADIENT> run;
            run.load(e, row, col);
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            const int64_t at = (int64_t)row * ld + col;
            if constexpr (IN == 2) {
                for (int s = 0; s < planes; s += 8) {
                    float w[8][4];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (s + u < planes) load_values<2>(in, (s + u) * plane_stride + at, e.N - col, w[u]);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (s + u < planes) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[i] += w[u][i];
                        }
                }
            } else {
                load_values<IN>(in, at, e.N - col, v);
            }
            run.finish(e, row, col, bias, v);
            if constexpr (GRADIENT) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[i] += v[i];
            }
        }
    }
    if constexpr (GRADIENT) {
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
}

// out[c] = sum of partials[i][c], i < count, in a fixed order: 32 threads take
// every 32nd partial of a column, four loads in flight, and their sums are
// added in thread order.  32 columns per block and turn.  125 x 500: 2.8 us
// against 6.9 with 8 threads per column (both mostly the launch and the loads'
// latency).
constexpr int kSumBlocks = 1 << 20;
__global__ __launch_bounds__(1024)
void column_sum_kernel(int count, int n, const float* partials, float* out) {
    __shared__ float part[32][33];
    const int tc = threadIdx.x % 32, tr = threadIdx.x / 32;
    for (int64_t first = 32 * (int64_t)blockIdx.x; first < n; first += 32 * (int64_t)gridDim.x) {
        const int64_t c = first + tc;
        float s = 0.f;
        if (c < n) {
            for (int i = tr; i < count; i += 128) {
                float v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] = i + 32 * u < count ? partials[(int64_t)(i + 32 * u) * n + c] : 0.f;
#pragma unroll
                for (int u = 0; u < 4; ++u) s += v[u];
            }
        }
        part[tr][tc] = s;
        __syncthreads();
        if (tr == 0 && c < n) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) t += part[i][tc];
            out[c] = t;
        }
        __syncthreads();                                     // part is read
    }
}

// Rows per block of the pass: enough blocks for the device's 256 CUs (eight
// each), then as many rows as that leaves, for fewer partial sums; a multiple
// of 8 between 8 and M, or the one above M (below 2^31: the largest M, 2^31 - 1,
// gives 2^31 - 8 and a second block of rows).
int pass_rows(int M, int N) {
    const int64_t cols = ceil_div(N, kPassCols);
    const int64_t rows = ((int64_t)M * cols + 2047) / 2048;
    const int64_t most = ((int64_t)M + 7) / 8 < INT_MAX / 8 ? ((int64_t)M + 7) / 8 : INT_MAX / 8;
    const int64_t eights = (rows + 7) / 8;
    return 8 * (int)(eights < 1 ? 1 : eights < most ? eights : most);
}

int64_t align256(int64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

hipError_t launch_column_sums(int count, int n, const float* partials, float* out, hipStream_t s) {
    const int blocks = ceil_div(n, 32);
    hipLaunchKernelGGL(column_sum_kernel, dim3(blocks < kSumBlocks ? blocks : kSumBlocks), dim3(1024), 0, s, count, n,
                       partials, out);
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
    auto launch = [&](auto in_c) {
        constexpr int IN = decltype(in_c)::value;
        if (e.gradient)
            hipLaunchKernelGGL((epilogue_kernel<IN, true>), grid, dim3(256), 0, s, e, in, ld, planes, plane_stride, rpb, part);
        else
            hipLaunchKernelGGL((epilogue_kernel<IN, false>), grid, dim3(256), 0, s, e, in, ld, planes, plane_stride, rpb, part);
    };
    if (in_type == 0) launch(std::integral_constant<int, 0>{});
    else if (in_type == 1) launch(std::integral_constant<int, 1>{});
    else launch(std::integral_constant<int, 2>{});
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || part == nullptr) return err;
    return launch_column_sums((int)gy, e.N, part, e.bias_grad, s);
}

namespace {

// ------------------------------------------------------- choice of kernel

enum { kRows = 0, kTiles = 1, kGeneral = 2 };
struct Plan {
    int kind;
    // kTiles: `tile` for the first `rows` rows of op(A) (all of them unless
    // split), rest_tile for the others
    int tile, rows, rest_tile;
    int splits;                               // kRows: blocks along K
    bool fused;                               // kRows: the fused kernel
    int k_share;                              // kTiles on 64 tiles: K per block, if below K
    bool pack_a, pack_b;                      // factors copied into the workspace
    int K;                                    // as the product runs it (padded if packed)
    int64_t lda, ldb;                         // of the copies, where packed
    int64_t a_bytes, b_bytes, main_bytes, part_rows;   // workspace: copies, planes, column sums
};

int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
// A factor of `rows` rows whose copies' 32-bit offsets hold, a tile's
// overhang included.
bool offsets_hold(int64_t rows, int64_t ld) { return ld < (1ll << 30) / (rows + 256); }

// Estimated time of an M x N x K product on `tile` x `tile` tiles, in us
// (MI355X, each kernel alone).  A round of 256 blocks takes the K loop,
// `slow` per 64-deep phase once all CUs are busy (`fast` up to half of them:
// the clock drops, and the small tiles' copies share the L2), and `fixed` for
// start and epilogue (with a kept pre-activation; the activation adds the
// same everywhere).  64 tiles: 4.4 and 0.0037 per k, but 0.0017 up to 16 of
// them whose factors are both mn-contiguous (the L2 has whole lines for those).
// 128 tiles copy k-contiguous factors in runs of 64 bytes: 0.06 more for each.  4096^3: 106 / 135 / 165 / 160 / 262
// us on 256 / 192 / 160 / 128 / 64 tiles; 1000 x 2000 x 1000: 41 / 26 / 22 / 21
// / 17.
double tile_time(int tile, int M, int N, int K, int k_contiguous) {
    const double tiles = (double)ceil_div(M, tile) * ceil_div(N, tile);
    const double rounds = ceil(tiles / 256.0);
    if (tile == 64) {
        const double shared = k_contiguous ? 1.0 : fmin(1.0, fmax(0.0, (tiles - 16.0) / 48.0));
        return rounds * (4.4 + (0.0017 + 0.0020 * shared) * K);
    }
    static const struct { int tile; double fast, slow, fixed; } kCost[] = {
        {256, 1.00, 1.38, 20.0}, {192, 0.70, 0.86, 13.0}, {160, 0.62, 0.70, 10.8}, {128, 0.31, 0.36, 16.0}};
    for (const auto& c : kCost)
        if (c.tile == tile) {
            const double busy = fmin(1.0, fmax(0.0, tiles / 128.0 - 1.0));
            const double slow = c.slow + (tile == 128 ? 0.06 * k_contiguous : 0.0);
            return rounds * ((c.fast + (slow - c.fast) * busy) * ceil_div(K, 64) + c.fixed);
        }
    return 1e30;
}

int pick_tile(int M, int N, int K, bool split_k, int k_contiguous, double* time) {
    int best = 256;
    *time = 1e30;
    for (const int tile : {256, 192, 160, 128, 64}) {
        if (tile <= 128 && !split_k) continue;
        const double t = tile_time(tile, M, N, K, k_contiguous);
        if (t < *time) {
            *time = t;
            best = tile;
        }
    }
    return best;
}

// Share of K per block on 64 tiles whose blocks split K, for few tiles and a
// long K: at most 256 blocks, shares of at least 256.  time: the product's,
// no less than its factors' read at 4.8 TB/s, and the pass's over the planes
// (from 5 us; 4 TB/s).  A small layer's weight gradient: 256 x 256 x 8192 11.5
// us against 18.3 unsplit, 512 x 512 x 8192 19 against 36; 24 x 8192 x 4096,
// bound by its weight's read, stays unsplit (16.5 against 18.1).
int pick_share(int M, int N, int K, double* time) {
    const int64_t tiles = (int64_t)ceil_div(M, 64) * ceil_div(N, 64);
    int64_t splits = 256 / tiles;
    if (splits > K / 256) splits = K / 256;
    *time = 1e30;
    if (splits < 2) return K;
    const int share = (ceil_div(K, (int)splits) + 63) / 64 * 64;
    const double product = fmax(4.4 + 0.0037 * share, 4.0 + 2.0 * ((double)M + N) * K / 4.8e6);
    *time = product + 5.0 + 8.0 * ceil_div(K, share) * (double)M * N / 4e6;
    return share;
}

// The estimates' choice among 64 tiles with K split over blocks and all
// tiles; fills q's tile, rows, rest_tile and k_share and returns the time.
double pick_product(int M, int N, int K, bool split_k, int k_contiguous, Plan* q) {
    double time;
    q->tile = pick_tile(M, N, K, split_k, k_contiguous, &time);
    q->rows = M;
    q->rest_tile = q->tile;
    q->k_share = K;
    // All rounds of 256 x 256 tiles but the last, the rows of that one on
    // smaller tiles.
    const int64_t tn = ceil_div(N, 256), tiles = ceil_div(M, 256) * tn, full = tiles / 256;
    const int64_t rows = full > 0 ? 256 * (256 * full / tn) : 0;
    if (rows > 0 && rows < M) {
        double rest;
        const int rest_tile = pick_tile(M - (int)rows, N, K, split_k, k_contiguous, &rest);
        const double top = tile_time(256, (int)rows, N, K, k_contiguous);
        if (top + rest < time) {
            time = top + rest;
            q->tile = 256;
            q->rows = (int)rows;
            q->rest_tile = rest_tile;
        }
    }
    if (split_k) {
        double split;
        const int share = pick_share(M, N, K, &split);
        if (split < time) {
            time = split;
            q->tile = q->rest_tile = 64;
            q->rows = M;
            q->k_share = share;
        }
    }
    return time;
}

Plan make_plan(const Gemm16Args& p, const EpilogueArgs& e, int op_a, int op_b) {
    Plan q{};
    q.K = p.K;
    q.lda = p.lda;
    q.ldb = p.ldb;
    // The tile kernels copy 4 bytes at a time at least: even leading
    // dimensions, widths of mn-contiguous factors, and K where a factor is
    // k-contiguous; the split-K ones 16 bytes along K.
    const bool both_mn = op_a && !op_b;
    const bool pad_k = !both_mn && p.K % 2 != 0;
    q.pack_a = pad_k || (reinterpret_cast<uintptr_t>(p.A) & 3) != 0 || p.lda % 2 != 0 || (op_a && p.M % 2 != 0);
    q.pack_b = pad_k || (reinterpret_cast<uintptr_t>(p.B) & 3) != 0 || p.ldb % 2 != 0 || (!op_b && p.N % 2 != 0);
    if (pad_k) q.K = (int)(pad8(p.K) > INT_MAX ? 0 : pad8(p.K));
    // Few rows, unless the weight is stored N x K and 64-column tiles fill
    // half the CUs: those copy it in whole cache lines (24 x 8192 x 4096: 16.5
    // us on 64 tiles, 20.9 on the few-row kernel; with N = 4096 12.6 against
    // 10.1 for one row).
    const bool tiles64 = op_b && p.N > 64 * 127 && p.K % 8 == 0 && !q.pack_a && !q.pack_b &&
                         offsets_hold(p.M, p.lda) && offsets_hold(p.N, p.ldb);
    if (p.M <= kLinearRowsMax && !op_a && p.K > 0 && p.K < (1 << 30) && !tiles64) {
        q.kind = kRows;
        q.K = p.K;
        q.pack_a = q.pack_b = false;
        q.splits = linear_rows_splits(p.M, p.N, p.K);
        q.fused = q.splits > 1 && !e.gradient && linear_rows_fused(p.M, p.N, p.K, op_b);
        if (q.fused) q.splits = 1;
        if (q.splits > 1 || e.gradient) q.main_bytes = align256(4 * (int64_t)q.splits * p.M * p.N);
        q.part_rows = e.bias_grad ? 1 : 0;
        return q;
    }
    const int kc = (op_a ? 0 : 1) + (op_b ? 1 : 0);
    double time = q.K > 0 ? pick_product(p.M, p.N, q.K, both_mn || q.K % 8 == 0, kc, &q) : 0.0;
    // K even but no multiple of 8 leaves the large tiles only: with few tiles
    // and a long K the copy into padded rows (from 4 us; 3 TB/s) and the split
    // of K cost less (395 x 72 x 2132: 12 us against 28).
    if (!both_mn && !pad_k && p.K % 8 != 0 && p.K < INT_MAX - 8) {
        Plan packed = q;
        packed.K = (int)pad8(p.K);
        const double copy = 4.0 + 4.0 * ((double)p.M + p.N) * packed.K / 3e6;
        if (copy + pick_product(p.M, p.N, packed.K, true, kc, &packed) < time) {
            q = packed;
            q.pack_a = q.pack_b = true;
        }
    }
    const int64_t a_rows = op_a ? q.K : p.M, b_rows = op_b ? p.N : q.K;
    if (q.pack_a) q.lda = pad8(op_a ? p.M : q.K);
    if (q.pack_b) q.ldb = pad8(op_b ? q.K : p.N);
    q.kind = kTiles;
    if (q.K == 0 || !offsets_hold(a_rows, q.lda) || !offsets_hold(b_rows, q.ldb)) {
        q.kind = kGeneral;
        q.pack_a = q.pack_b = false;
        q.main_bytes = align256(4 * (int64_t)p.M * p.N);
        q.part_rows = e.bias_grad ? 1 : 0;
        return q;
    }
    if (q.pack_a) q.a_bytes = align256(2 * a_rows * q.lda);
    if (q.pack_b) q.b_bytes = align256(2 * b_rows * q.ldb);
    if (q.k_share < q.K) q.main_bytes = align256(4 * (int64_t)ceil_div(q.K, q.k_share) * p.M * p.N);
    if (e.bias_grad)
        q.part_rows = ceil_div(q.rows, q.tile) + (q.rows < p.M ? ceil_div(p.M - q.rows, q.rest_tile) : 0);
    return q;
}

int64_t sums_bytes(const Plan& q, const EpilogueArgs& e) {
    if (!e.bias_grad) return 0;
    return q.kind == kTiles && q.k_share == q.K ? align256(4 * q.part_rows * e.N) : epilogue_pass_workspace(e.M, e.N);
}

// rows x cols 16-bit values (leading dimension ld_in, any alignment) into
// out_rows x ld_out ones, zeros around them; block row y < blocks_a is the
// first factor's.
struct PackArgs {
    const uint16_t* in; int64_t ld_in;
    uint16_t* out; int64_t ld_out;
    int rows, cols, out_rows;
};
__global__ __launch_bounds__(256)
void pack_kernel(PackArgs a, PackArgs b, int blocks_a) {
    const bool second = (int)blockIdx.y >= blocks_a;
    const PackArgs& m = second ? b : a;
    const int64_t first = (second ? blockIdx.y - blocks_a : blockIdx.y), step = second ? gridDim.y - blocks_a : blocks_a;
    const int chunks = (int)(m.ld_out / 8);
    const int64_t total = (int64_t)m.out_rows * chunks;
    for (int64_t i = first * 256 + threadIdx.x; i < total; i += step * 256) {
        const int r = (int)(i / chunks), c = 8 * (int)(i - (int64_t)r * chunks);
        uint16_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (r < m.rows && c < m.cols) {
            const uint16_t* q = m.in + (int64_t)r * m.ld_in + c;
            if (c + 8 <= m.cols) {
                __builtin_memcpy(v, q, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < m.cols) v[e] = q[e];
            }
        }
        __builtin_memcpy(m.out + (int64_t)r * m.ld_out + c, v, 16);
    }
}

hipError_t launch_tiles(int tile, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a,
                        int op_b, float* partials) {
    switch (tile) {
        case 256: return launch_linear_wide256(p, e, s, format, op_a, op_b, partials);
        case 192: return launch_linear_wide192(p, e, s, format, op_a, op_b, partials);
        case 160: return launch_linear_wide160(p, e, s, format, op_a, op_b, partials);
        case 128: return launch_linear_ksplit128(p, e, s, format, op_a, op_b, partials);
        default: return launch_linear_ksplit(p, e, s, format, op_a, op_b, partials);
    }
}

// The epilogue of the rows from `row` on.
EpilogueArgs rows_from(const EpilogueArgs& e, int row) {
    EpilogueArgs r = e;
    const int64_t size = e.c_type == 2 ? 4 : 2;
    r.M = e.M - row;
    r.C = static_cast<char*>(e.C) + size * row * e.ldc;
    if (e.residual) r.residual = static_cast<const char*>(e.residual) + size * row * e.ldr;
    if (e.preact) r.preact = static_cast<char*>(e.preact) + 2 * row * e.ldz;
    return r;
}

}  // namespace

int64_t linear_workspace(const Gemm16Args& p, const EpilogueArgs& e, int op_a, int op_b) {
    const Plan q = make_plan(p, e, op_a, op_b);
    return q.a_bytes + q.b_bytes + q.main_bytes + sums_bytes(q, e);
}

hipError_t launch_linear(const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_a, int op_b,
                         void* workspace) {
    const Plan q = make_plan(p, e, op_a, op_b);
    char* const ws = static_cast<char*>(workspace);
    uint16_t* const a_copy = reinterpret_cast<uint16_t*>(ws);
    uint16_t* const b_copy = reinterpret_cast<uint16_t*>(ws + q.a_bytes);
    float* const main = reinterpret_cast<float*>(ws + q.a_bytes + q.b_bytes);
    float* const partials = reinterpret_cast<float*>(ws + q.a_bytes + q.b_bytes + q.main_bytes);
    hipError_t err;
    if (q.kind == kRows) {
        if (q.fused) return launch_linear_rows_fused(p, e, s, format, op_b);
        const bool planes = q.splits > 1 || e.gradient;
        err = launch_linear_rows(p, e, s, format, op_b, q.splits, planes ? main : nullptr);
        if (err != hipSuccess || !planes) return err;
        return launch_epilogue_pass(e, 2, main, p.N, q.splits, (int64_t)p.M * p.N, partials, s);
    }
    if (q.kind == kGeneral) {
        Gemm16Args r = p;
        r.C = main;
        r.ldc = p.N;
        err = (op_a || op_b) ? launch_mixed_op(r, s, format, op_a, op_b)
                             : launch_mixed(r, s, format, mixed_pick_config(r.M, r.N, r.K));
        if (err != hipSuccess) return err;
        return launch_epilogue_pass(e, 2, main, p.N, 1, 0, partials, s);
    }
    Gemm16Args r = p;
    r.K = q.K;
    if (q.pack_a || q.pack_b) {
        const PackArgs a{p.A, p.lda, a_copy, q.lda, op_a ? p.K : p.M, op_a ? p.M : p.K, op_a ? q.K : p.M};
        const PackArgs b{p.B, p.ldb, b_copy, q.ldb, op_b ? p.N : p.K, op_b ? p.K : p.N, op_b ? p.N : q.K};
        auto blocks = [](const PackArgs& m) {
            const int64_t n = ((int64_t)m.out_rows * (m.ld_out / 8) + 255) / 256;
            return (int)(n > 1024 ? 1024 : n);
        };
        const int ba = q.pack_a ? blocks(a) : 0, bb = q.pack_b ? blocks(b) : 0;
        hipLaunchKernelGGL(pack_kernel, dim3(1, (unsigned)(ba + bb)), dim3(256), 0, s, a, b, ba);
        if ((err = hipGetLastError()) != hipSuccess) return err;
        if (q.pack_a) {
            r.A = a_copy;
            r.lda = q.lda;
        }
        if (q.pack_b) {
            r.B = b_copy;
            r.ldb = q.ldb;
        }
    }
    // An odd width of an mn-contiguous factor (then packed, zeros beside it)
    // goes to the product as the even one above: its copies' range ends on a
    // dword.  The epilogue keeps to e.M and e.N.
    if (op_a) r.M = p.M + p.M % 2;
    if (!op_b) r.N = p.N + p.N % 2;
    if (q.k_share < q.K) {
        err = launch_linear_ksplit_planes(r, e.M, e.N, s, format, op_a, op_b, q.k_share, main);
        if (err != hipSuccess) return err;
        return launch_epilogue_pass(e, 2, main, p.N, ceil_div(q.K, q.k_share), (int64_t)p.M * p.N, partials, s);
    }
    float* const part = e.bias_grad ? partials : nullptr;
    const bool split = q.rows < p.M;
    Gemm16Args top = r;
    EpilogueArgs te = e;
    if (split) top.M = te.M = q.rows;
    err = launch_tiles(q.tile, top, te, s, format, op_a, op_b, part);
    if (err == hipSuccess && split) {
        Gemm16Args rest = r;
        rest.M = r.M - q.rows;
        rest.A = r.A + (op_a ? (int64_t)q.rows : (int64_t)q.rows * r.lda);
        err = launch_tiles(q.rest_tile, rest, rows_from(e, q.rows), s, format, op_a, op_b,
                           part ? part + (int64_t)ceil_div(q.rows, q.tile) * p.N : nullptr);
    }
    if (err != hipSuccess || part == nullptr) return err;
    return launch_column_sums((int)q.part_rows, p.N, part, e.bias_grad, s);
}

}  // namespace gemmf32
