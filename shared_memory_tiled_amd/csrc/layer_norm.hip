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
//
// Bound by memory: forward one read and one write of the matrix, backward two
// (three) reads and one write.  A row stays in registers between its passes:
// `THREADS` threads hold it in CH chunks of 16 bytes each, a wave, a block of
// 256 or one of 1024 by its length, and the parameters stay in registers from
// row to row (blocks walk the rows).  Rows longer than a block's registers go
// through the kernels at the end, which read them again.
//
// The binary32 sum of a row rounds, so its mean m is off by a few units of the
// row's size, even where all values are equal: up to 2.5e-7 of 4096 of them,
// which a row constant at 1000 would turn into 0.08 at rstd = 316.  A second
// reduction therefore takes the deviations d = x - m, which are exact where the
// row is near its mean, both squared and as they are: delta = <d> is what m
// lacks, the deviations become d - delta, the mean m + delta, and
// <(d - delta)^2> = <d^2> - delta^2.  Where delta^2 is more than 2^-6 of <d^2>
// (rows as good as constant) that difference cancels, and the squares are
// taken again.
#include "epilogue.h"

namespace gemmf32 {

namespace {

template <int TYPE>
constexpr int kChunk = TYPE == 2 ? 4 : 8;                 // values per 16 bytes

__device__ __forceinline__ float wave_total(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
// The sum of v over THREADS threads (a wave, or the whole block) in each of
// them; slots: one float per wave.
template <int THREADS>
__device__ __forceinline__ float group_total(float v, float* slots) {
    v = wave_total(v);
    if constexpr (THREADS > 64) {
        __syncthreads();                                  // the slots' last readers are done
        if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
        __syncthreads();
        v = slots[0];
#pragma unroll
        for (int i = 1; i < THREADS / 64; ++i) v += slots[i];
    }
    return v;
}

// Two sums at once, with one pair of barriers; slots: two floats per wave.
template <int THREADS>
__device__ __forceinline__ void group_totals(float& v, float& w, float* slots) {
    v = wave_total(v);
    w = wave_total(w);
    if constexpr (THREADS > 64) {
        __syncthreads();                                  // the slots' last readers are done
        if ((threadIdx.x & 63) == 0) {
            slots[2 * (threadIdx.x >> 6)] = v;
            slots[2 * (threadIdx.x >> 6) + 1] = w;
        }
        __syncthreads();
        v = slots[0];
        w = slots[1];
#pragma unroll
        for (int i = 1; i < THREADS / 64; ++i) {
            v += slots[2 * i];
            w += slots[2 * i + 1];
        }
    }
}
// Whether the squares' mean has to be taken again about the corrected mean
// (the same in every thread of a row; false for NaN).
__device__ __forceinline__ bool near_constant(float delta, float square) { return delta * delta > 0.015625f * square; }

// The corrected mean; m itself for rows with infinities.
__device__ __forceinline__ float corrected(float m, float delta) {
    return __builtin_fabsf(delta) < __builtin_inff() ? m + delta : m;
}

// A 16-byte chunk that exists in whole, as loaded, and its values.
typedef unsigned chunk_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ chunk_t load_raw(const char* row, int byte) {
    chunk_t v;
    __builtin_memcpy(&v, row + byte, 16);
    return v;
}
template <int TYPE>
__device__ __forceinline__ void unpack(chunk_t raw, float (&v)[kChunk<TYPE>]) {
    typename Stored<TYPE>::T t[kChunk<TYPE>];
    __builtin_memcpy(t, &raw, 16);
#pragma unroll
    for (int e = 0; e < kChunk<TYPE>; ++e) v[e] = (float)t[e];
}
// One 16-byte chunk of a row from column c (zeros from column `cols` on), as
// binary32.
template <int TYPE>
__device__ __forceinline__ void load_chunk(const void* row, int c, int cols, float (&v)[kChunk<TYPE>]) {
    if (c < cols) {
        load_values<TYPE>(row, c, cols - c, v);
    } else {
#pragma unroll
        for (int e = 0; e < kChunk<TYPE>; ++e) v[e] = 0.0f;
    }
}
template <int TYPE, int CH>
__device__ __forceinline__ void load_params(const LayerNormArgs& a, const void* p, float missing, int t, int threads,
                                            float (&v)[CH][kChunk<TYPE>]) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const int c = kChunk<TYPE> * (t + k * threads);
#pragma unroll
        for (int e = 0; e < kChunk<TYPE>; ++e) v[k][e] = missing;
        if (p != nullptr && c < a.cols) load_values(a.param_type, p, c, a.cols - c, v[k]);
    }
}
template <int TYPE>
__device__ __forceinline__ const char* row_of(const void* base, int64_t row, int64_t ld) {
    return static_cast<const char*>(base) + (TYPE == 2 ? 4 : 2) * row * ld;
}

// FIT: how the row fills its chunks.
//   kWhole   every chunk (cols = THREADS CH V): no access is conditional, and
//            the next row's loads are in flight while this one is worked on
//            (a wait for them need not wait for the stores after them, which
//            the same counter counts).  8192^2 bf16: 56 us, 81 without.
//   kChunks  whole chunks, some missing (cols a multiple of V): the same, with
//            missing chunks' loads repeating the last one's
//   kRagged  the last chunk in part: loads where they are used
enum { kWhole, kChunks, kRagged };
template <int TYPE, int THREADS, int CH, int FIT>
__global__ __launch_bounds__(THREADS == 1024 ? 1024 : 256)
void layer_norm_kernel(LayerNormArgs a) {
    constexpr int V = kChunk<TYPE>, BLOCK = THREADS == 1024 ? 1024 : 256, GROUPS = BLOCK / THREADS;
    __shared__ float slots[2 * (BLOCK / 64)];
    const int t = threadIdx.x % THREADS, g = threadIdx.x / THREADS;
    float gamma[CH][V], beta[CH][V];
    load_params<TYPE>(a, a.gamma, 1.0f, t, THREADS, gamma);
    load_params<TYPE>(a, a.beta, 0.0f, t, THREADS, beta);
    const float inv = 1.0f / (float)a.cols;
    const int64_t step = (int64_t)gridDim.x * GROUPS;
    int64_t row = (int64_t)blockIdx.x * GROUPS + g;
    chunk_t next[CH];
    const int chunks = a.cols / V;
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
        const char* const x = row_of<TYPE>(a.x, r, a.ldx);
#pragma unroll
        for (int k = 0; k < CH; ++k)
            next[k] = load_raw(x, 16 * (FIT == kWhole ? t + k * THREADS : min(t + k * THREADS, chunks - 1)));
    };
    if constexpr (FIT != kRagged) fetch(row < a.rows ? row : a.rows - 1);
    for (; row < a.rows; row += step) {
        float v[CH][V];
        float s = 0.0f;
        if constexpr (FIT != kRagged) {
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                unpack<TYPE>(next[k], v[k]);
                if (FIT == kChunks && t + k * THREADS >= chunks) {
#pragma unroll
                    for (int e = 0; e < V; ++e) v[k][e] = 0.0f;
                }
            }
            fetch(row + step < a.rows ? row + step : row);
        } else {
            const char* const x = row_of<TYPE>(a.x, row, a.ldx);
#pragma unroll
            for (int k = 0; k < CH; ++k) load_chunk<TYPE>(x, V * (t + k * THREADS), a.cols, v[k]);
        }
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) s += v[k][e];
        const float m = group_total<THREADS>(s, slots) / (float)a.cols;
        auto inside = [&](int k, int e) __attribute__((always_inline)) {
            return FIT == kWhole || V * (t + k * THREADS) + e < a.cols;
        };
        float delta = 0.0f, square = 0.0f;
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = inside(k, e) ? v[k][e] - m : 0.0f;
                v[k][e] = d;
                delta += d;
                square = __builtin_fmaf(d, d, square);
            }
        group_totals<THREADS>(delta, square, slots);
        delta *= inv;
        square *= inv;
        float var = __builtin_fmaf(-delta, delta, square);
        if (near_constant(delta, square)) {
            s = 0.0f;
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = inside(k, e) ? v[k][e] - delta : 0.0f;
                    s = __builtin_fmaf(d, d, s);
                }
            var = group_total<THREADS>(s, slots) * inv;
        }
        const float mean = corrected(m, delta), rstd = 1.0f / sqrtf(var + a.eps);
        const float shift = -delta * rstd;
        char* const y = const_cast<char*>(row_of<TYPE>(a.y, row, a.ldy));
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = V * (t + k * THREADS);
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[k][e] = __builtin_fmaf(__builtin_fmaf(v[k][e], rstd, shift), gamma[k][e], beta[k][e]);
            if (FIT == kWhole || c < a.cols) store_values<TYPE>(y, c, FIT != kRagged ? V : a.cols - c, v[k]);
        }
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// Blocks of 512 threads (256 registers each: the sums of a chunk's columns,
// its parameters, the row and the next one's loads), GROUPS rows at a time; block b takes rows b GROUPS
// .., then gridDim.x GROUPS further, and leaves its sums for dgamma and dbeta
// in row b of `partials` (2 cols floats: dgamma's, then dbeta's).
template <int TYPE, int THREADS, int CH, int FIT>
__global__ __launch_bounds__(512)
void layer_norm_backward_kernel(LayerNormArgs a, float* partials) {
    constexpr int V = kChunk<TYPE>, GROUPS = 512 / THREADS, WAVES = THREADS / 64;
    constexpr int COLS = THREADS * CH * V;
    __shared__ float slots[2][8][2];
    __shared__ float sums[GROUPS > 1 ? (GROUPS - 1) * COLS : 1];
    const int t = threadIdx.x % THREADS, g = threadIdx.x / THREADS, wave = threadIdx.x >> 6;
    float gamma[CH][V], dg[CH][V], db[CH][V];
    load_params<TYPE>(a, a.gamma, 1.0f, t, THREADS, gamma);
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) dg[k][e] = db[k][e] = 0.0f;
    const float inv = 1.0f / (float)a.cols;
    int parity = 0;
    // FIT as for layer_norm_kernel; the next rows' loads, a turn ahead.
    const int chunks = a.cols / V;
    chunk_t next_x[CH], next_dy[CH], next_r[CH];
    auto row_at = [&](int64_t first) __attribute__((always_inline)) {
        return first + g < a.rows ? first + g : a.rows - 1;
    };
    auto fetch = [&](chunk_t (&next)[CH], const void* base, int64_t first, int64_t ld) __attribute__((always_inline)) {
        const char* const r = row_of<TYPE>(base, row_at(first), ld);
#pragma unroll
        for (int k = 0; k < CH; ++k)
            next[k] = load_raw(r, 16 * (FIT == kWhole ? t + k * THREADS : min(t + k * THREADS, chunks - 1)));
    };
    if constexpr (FIT != kRagged) {
        fetch(next_x, a.x, (int64_t)blockIdx.x * GROUPS, a.ldx);
        fetch(next_dy, a.dy, (int64_t)blockIdx.x * GROUPS, a.lddy);
        if (a.residual_grad) fetch(next_r, a.residual_grad, (int64_t)blockIdx.x * GROUPS, a.ldr);
    }
    // every group makes the same number of turns (the barrier is the block's)
    for (int64_t first = (int64_t)blockIdx.x * GROUPS; first < a.rows; first += (int64_t)gridDim.x * GROUPS) {
        const int64_t row = first + g;
        const bool inside = row < a.rows;
        const char* const xr = row_of<TYPE>(a.x, row, a.ldx);
        const char* const dyr = row_of<TYPE>(a.dy, row, a.lddy);
        const int cols = inside ? a.cols : 0;
        float xhat[CH][V], gy[CH][V];
        float s0 = 0.0f, s1 = 0.0f;
        const float mean = inside ? a.mean[row] : 0.0f, rstd = inside ? a.rstd[row] : 0.0f;
        const int64_t after = first + (int64_t)gridDim.x * GROUPS;
        if constexpr (FIT != kRagged) {
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                unpack<TYPE>(next_x[k], xhat[k]);
                unpack<TYPE>(next_dy[k], gy[k]);
                if (FIT == kChunks && t + k * THREADS >= chunks) {
#pragma unroll
                    for (int e = 0; e < V; ++e) xhat[k][e] = gy[k][e] = 0.0f;
                }
            }
            fetch(next_x, a.x, after < a.rows ? after : first, a.ldx);
            fetch(next_dy, a.dy, after < a.rows ? after : first, a.lddy);
            if (!inside) {                                          // the last row again: not counted
#pragma unroll
                for (int k = 0; k < CH; ++k)
#pragma unroll
                    for (int e = 0; e < V; ++e) xhat[k][e] = gy[k][e] = 0.0f;
            }
        } else {
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const int c = V * (t + k * THREADS);
                load_chunk<TYPE>(xr, c, cols, xhat[k]);
                load_chunk<TYPE>(dyr, c, cols, gy[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                xhat[k][e] = (xhat[k][e] - mean) * rstd;            // dy past the row's end is zero
                const float d = gy[k][e];
                dg[k][e] = __builtin_fmaf(d, xhat[k][e], dg[k][e]);
                db[k][e] += d;
                gy[k][e] = d * gamma[k][e];
                s0 += gy[k][e];
                s1 = __builtin_fmaf(gy[k][e], xhat[k][e], s1);
            }
        }
        s0 = wave_total(s0);
        s1 = wave_total(s1);
        if constexpr (WAVES > 1) {
            if ((threadIdx.x & 63) == 0) {
                slots[parity][wave][0] = s0;
                slots[parity][wave][1] = s1;
            }
            __syncthreads();
            s0 = s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) {
                s0 += slots[parity][g * WAVES + i][0];
                s1 += slots[parity][g * WAVES + i][1];
            }
            parity ^= 1;
        }
        s0 *= inv;
        s1 *= inv;
        const char* const rr = row_of<TYPE>(a.residual_grad, row, a.ldr);
        char* const dxr = const_cast<char*>(row_of<TYPE>(a.dx, row, a.lddx));
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = V * (t + k * THREADS);
            if (FIT == kWhole ? !inside : c >= cols) continue;
            float r[V];
#pragma unroll
            for (int e = 0; e < V; ++e) r[e] = 0.0f;
            if (a.residual_grad) {
                if constexpr (FIT != kRagged) unpack<TYPE>(next_r[k], r);
                else load_chunk<TYPE>(rr, c, cols, r);
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                r[e] = __builtin_fmaf(rstd, gy[k][e] - s0 - xhat[k][e] * s1, r[e]);
            store_values<TYPE>(dxr, c, FIT != kRagged ? V : cols - c, r);
        }
        if (FIT != kRagged && a.residual_grad) fetch(next_r, a.residual_grad, after < a.rows ? after : first, a.ldr);
    }
    if (partials == nullptr) return;
    // The groups' sums, in group order; then the block's row of partials.
    float* const out = partials + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        auto& acc = which == 0 ? dg : db;
        if constexpr (GROUPS > 1) {
            __syncthreads();
            if (g > 0) {
#pragma unroll
                for (int k = 0; k < CH; ++k)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        sums[(g - 1) * COLS + V * (t + k * THREADS) + e] = acc[k][e];
            }
            __syncthreads();
            if (g == 0) {
#pragma unroll
                for (int k = 0; k < CH; ++k)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        for (int i = 0; i < GROUPS - 1; ++i)
                            acc[k][e] += sums[i * COLS + V * (t + k * THREADS) + e];
            }
        }
        if (g == 0) {
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const int c = V * (t + k * THREADS);
                if (c < a.cols) store_values<2>(out, (int64_t)which * a.cols + c, a.cols - c, acc[k]);
            }
        }
    }
}

// dgamma and dbeta from `count` rows of partials, in a fixed order: 32
// threads per column take every 32nd, their sums are added in thread order.
__global__ __launch_bounds__(1024)
void param_grad_kernel(int count, int cols, const float* partials, float* dgamma, float* dbeta) {
    __shared__ float part[32][33];
    float* const out = blockIdx.y == 0 ? dgamma : dbeta;
    if (out == nullptr) return;                           // the same for the whole block
    const int tc = threadIdx.x % 32, tr = threadIdx.x / 32, c = blockIdx.x * 32 + tc;
    float s = 0.0f;
    if (c < cols)
        for (int i = tr; i < count; i += 32) s += partials[((int64_t)2 * i + blockIdx.y) * cols + c];
    part[tr][tc] = s;
    __syncthreads();
    if (tr == 0 && c < cols) {
        float t = 0.0f;
        for (int i = 0; i < 32; ++i) t += part[i][tc];
        out[c] = t;
    }
}

// ------------------------------------------------------ rows of any length

constexpr int kThreads = 256;

template <int TYPE>
__global__ __launch_bounds__(kThreads)
void layer_norm_long_kernel(LayerNormArgs a) {
    constexpr int V = kChunk<TYPE>;
    __shared__ float slots[8];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* const x = row_of<TYPE>(a.x, row, a.ldx);
        char* const y = const_cast<char*>(row_of<TYPE>(a.y, row, a.ldy));
        float s = 0.0f;
        for (int64_t c = V * threadIdx.x; c < a.cols; c += V * kThreads) {
            float v[V];
            load_chunk<TYPE>(x, (int)c, a.cols, v);
#pragma unroll
            for (int e = 0; e < V; ++e) s += v[e];
        }
        const float m = group_total<kThreads>(s, slots) / (float)a.cols;
        // the sums of x - m - shift and of its square
        auto deviations = [&](float shift, float& sum, float& square) __attribute__((always_inline)) {
            sum = square = 0.0f;
            for (int64_t c = V * threadIdx.x; c < a.cols; c += V * kThreads) {
                float v[V];
                load_chunk<TYPE>(x, (int)c, a.cols, v);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = c + e < a.cols ? v[e] - m - shift : 0.0f;
                    sum += d;
                    square = __builtin_fmaf(d, d, square);
                }
            }
            group_totals<kThreads>(sum, square, slots);
        };
        float delta, square;
        deviations(0.0f, delta, square);
        delta /= (float)a.cols;
        square /= (float)a.cols;
        float var = __builtin_fmaf(-delta, delta, square);
        if (near_constant(delta, square)) {
            float left;
            deviations(delta, left, square);
            var = square / (float)a.cols;
        }
        const float mean = corrected(m, delta), rstd = 1.0f / sqrtf(var + a.eps);
        for (int64_t c = V * threadIdx.x; c < a.cols; c += V * kThreads) {
            float v[V], g[V], b[V];
            load_chunk<TYPE>(x, (int)c, a.cols, v);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                g[e] = 1.0f;
                b[e] = 0.0f;
            }
            const int valid = a.cols - (int)c;
            if (a.gamma) load_values(a.param_type, a.gamma, c, valid, g);
            if (a.beta) load_values(a.param_type, a.beta, c, valid, b);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = __builtin_fmaf((v[e] - m - delta) * rstd, g[e], b[e]);
            store_values<TYPE>(y, c, valid, v);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

template <int TYPE>
__global__ __launch_bounds__(kThreads)
void layer_norm_backward_long_kernel(LayerNormArgs a) {
    constexpr int V = kChunk<TYPE>;
    __shared__ float slots[4];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* const xr = row_of<TYPE>(a.x, row, a.ldx);
        const char* const dyr = row_of<TYPE>(a.dy, row, a.lddy);
        const char* const rr = row_of<TYPE>(a.residual_grad, row, a.ldr);
        char* const dxr = const_cast<char*>(row_of<TYPE>(a.dx, row, a.lddx));
        const float mean = a.mean[row], rstd = a.rstd[row];
        // xhat and g = dy gamma of the chunk at c
        auto chunk = [&](int64_t c, float (&xhat)[V], float (&g)[V]) __attribute__((always_inline)) {
            load_chunk<TYPE>(xr, (int)c, a.cols, xhat);
            load_chunk<TYPE>(dyr, (int)c, a.cols, g);
            if (a.gamma) {
                float p[V];
                load_values(a.param_type, a.gamma, c, a.cols - (int)c, p);
#pragma unroll
                for (int e = 0; e < V; ++e) g[e] *= p[e];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) xhat[e] = (xhat[e] - mean) * rstd;
        };
        float s0 = 0.0f, s1 = 0.0f;
        for (int64_t c = V * threadIdx.x; c < a.cols; c += V * kThreads) {
            float xhat[V], g[V];
            chunk(c, xhat, g);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s0 += g[e];
                s1 = __builtin_fmaf(g[e], xhat[e], s1);
            }
        }
        const float m0 = group_total<kThreads>(s0, slots) / (float)a.cols;
        const float m1 = group_total<kThreads>(s1, slots) / (float)a.cols;
        for (int64_t c = V * threadIdx.x; c < a.cols; c += V * kThreads) {
            float xhat[V], g[V], r[V];
            chunk(c, xhat, g);
#pragma unroll
            for (int e = 0; e < V; ++e) r[e] = 0.0f;
            if (a.residual_grad) load_chunk<TYPE>(rr, (int)c, a.cols, r);
#pragma unroll
            for (int e = 0; e < V; ++e) r[e] = __builtin_fmaf(rstd, g[e] - m0 - xhat[e] * m1, r[e]);
            store_values<TYPE>(dxr, c, a.cols - (int)c, r);
        }
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

// dx may be dy, so the column sums come first.
template <int TYPE>
hipError_t launch_long_backward(const LayerNormArgs& a, void* workspace, hipStream_t s) {
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
    const int64_t rows = a.rows < (1 << 22) ? a.rows : (1 << 22);
    hipLaunchKernelGGL(layer_norm_backward_long_kernel<TYPE>, dim3((unsigned)rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

// ------------------------------------------------------------- launchers

// Blocks that walk the rows: enough to fill the device (2048 threads per CU).
unsigned walkers(int64_t rows, int groups, int per_device) {
    const int64_t blocks = (rows + groups - 1) / groups;
    return (unsigned)(blocks < per_device ? blocks : per_device);
}

template <int TYPE, int THREADS, int CH>
hipError_t launch_forward(const LayerNormArgs& a, hipStream_t s) {
    constexpr int BLOCK = THREADS == 1024 ? 1024 : 256;
    const dim3 grid(walkers(a.rows, BLOCK / THREADS, 256 * 2048 / BLOCK));
    if (a.cols == THREADS * CH * kChunk<TYPE>)
        hipLaunchKernelGGL((layer_norm_kernel<TYPE, THREADS, CH, kWhole>), grid, dim3(BLOCK), 0, s, a);
    else if (a.cols % kChunk<TYPE> == 0)
        hipLaunchKernelGGL((layer_norm_kernel<TYPE, THREADS, CH, kChunks>), grid, dim3(BLOCK), 0, s, a);
    else
        hipLaunchKernelGGL((layer_norm_kernel<TYPE, THREADS, CH, kRagged>), grid, dim3(BLOCK), 0, s, a);
    return hipGetLastError();
}
template <int TYPE>
hipError_t forward(const LayerNormArgs& a, hipStream_t s) {
    const int64_t chunks = ((int64_t)a.cols + kChunk<TYPE> - 1) / kChunk<TYPE>;
    if (chunks <= 64) return launch_forward<TYPE, 64, 1>(a, s);
    if (chunks <= 128) return launch_forward<TYPE, 64, 2>(a, s);
    if (chunks <= 256) return launch_forward<TYPE, 256, 1>(a, s);
    if (chunks <= 512) return launch_forward<TYPE, 256, 2>(a, s);
    if (chunks <= 1024) return launch_forward<TYPE, 256, 4>(a, s);
    if (chunks <= 2048) return launch_forward<TYPE, 1024, 2>(a, s);
    if constexpr (TYPE == 2)                              // 16 values of 16 bits a thread fill its registers
        if (chunks <= 4096) return launch_forward<TYPE, 1024, 4>(a, s);
    const int64_t rows = a.rows < (1 << 22) ? a.rows : (1 << 22);
    hipLaunchKernelGGL(layer_norm_long_kernel<TYPE>, dim3((unsigned)rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

constexpr int kBackwardBlocks = 256;
constexpr int64_t kBackwardChunks = 2048;                 // per row, in registers

template <int TYPE, int THREADS, int CH>
hipError_t launch_backward(const LayerNormArgs& a, float* partials, hipStream_t s) {
    const unsigned blocks = walkers(a.rows, 512 / THREADS, kBackwardBlocks);
    const dim3 grid(blocks), block(512);
    // 32 columns a thread leave no registers for the next row's loads
    constexpr bool kAhead = CH * kChunk<TYPE> < 32;
    if (kAhead && a.cols == THREADS * CH * kChunk<TYPE>)
        hipLaunchKernelGGL((layer_norm_backward_kernel<TYPE, THREADS, CH, kAhead ? kWhole : kRagged>), grid, block, 0, s,
                           a, partials);
    else if (kAhead && a.cols % kChunk<TYPE> == 0)
        hipLaunchKernelGGL((layer_norm_backward_kernel<TYPE, THREADS, CH, kAhead ? kChunks : kRagged>), grid, block, 0,
                           s, a, partials);
    else
        hipLaunchKernelGGL((layer_norm_backward_kernel<TYPE, THREADS, CH, kRagged>), grid, block, 0, s, a, partials);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || partials == nullptr) return e;
    hipLaunchKernelGGL(param_grad_kernel, dim3(ceil_div(a.cols, 32), 2), dim3(1024), 0, s, (int)blocks, a.cols,
                       partials, a.dgamma, a.dbeta);
    return hipGetLastError();
}
template <int TYPE>
hipError_t backward(const LayerNormArgs& a, void* workspace, hipStream_t s) {
    const int64_t chunks = ((int64_t)a.cols + kChunk<TYPE> - 1) / kChunk<TYPE>;
    float* const partials = a.dgamma != nullptr || a.dbeta != nullptr ? static_cast<float*>(workspace) : nullptr;
    if (chunks <= 64) return launch_backward<TYPE, 64, 1>(a, partials, s);
    if (chunks <= 128) return launch_backward<TYPE, 64, 2>(a, partials, s);
    if (chunks <= 256) return launch_backward<TYPE, 256, 1>(a, partials, s);
    if (chunks <= 512) return launch_backward<TYPE, 256, 2>(a, partials, s);
    if (chunks <= 1024) return launch_backward<TYPE, 512, 2>(a, partials, s);
    if (chunks <= kBackwardChunks) return launch_backward<TYPE, 512, 4>(a, partials, s);
    return launch_long_backward<TYPE>(a, workspace, s);
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s) {
    if (a.type == 0) return forward<0>(a, s);
    if (a.type == 1) return forward<1>(a, s);
    return forward<2>(a, s);
}

int64_t layer_norm_backward_workspace(int type, int64_t rows, int cols) {
    const int chunk = type == 2 ? 4 : 8;
    const int64_t chunks = ((int64_t)cols + chunk - 1) / chunk;
    const int64_t blocks = chunks <= kBackwardChunks ? (rows < kBackwardBlocks ? rows : kBackwardBlocks)
                                                     : column_blocks(rows);
    return 2 * 4 * blocks * cols;
}

hipError_t launch_layer_norm_backward(const LayerNormArgs& a, void* workspace, hipStream_t s) {
    if (a.type == 0) return backward<0>(a, workspace, s);
    if (a.type == 1) return backward<1>(a, workspace, s);
    return backward<2>(a, workspace, s);
}

}  // namespace gemmf32
