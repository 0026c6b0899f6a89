// grad_norm.hip -- the norm over all of a model's gradients, and their
// clipping.
//
//   norm = sqrt(sum over tensors and values of g^2)
//   g <- g min(1, max_norm / (norm + eps))
//
// Two passes over the gradients, for the factor is known only after the whole
// sum; both are bound by memory.  A launch takes up to kGradTensors tensors,
// whose places travel in the kernel's arguments (no table in device memory to
// fill first, and a captured graph holds it).  Their values are dealt to the
// blocks in chunks of kGradChunk, a contiguous run of chunks to each, so that
// tensors of any sizes share the chip evenly.
//
// Squares are added in binary64, which holds every binary32 square: no value
// overflows or vanishes, and the order of adding does not show in the
// binary32 result.  Each block leaves one partial sum; partials are added in a
// fixed order, without atomics.  For the norm alone one block adds them; when both
// are asked for and the tensors fit one launch, every block of the second pass
// does so for itself (at most 16 KB from the L2 against a launch of its own: 41
// tensors of 9000 values 7.7 us against 8.5).  More launches would each read the
// partials of all of them in every block, a cost that grows with the square of
// their number (5000 tensors of 65536 values 4.26 ms against 0.77, 161 25.5 us
// against 23.7), so there the one block's launch comes between the passes.
//
// Roundings: the norm and the factor to binary32, a value times the factor to
// binary32 and, if its type is shorter, again to that (together up to 2^-24 of
// the value more than half a step of the type).
//
// Measured: 0.82e9 bf16 values in 161 tensors, into other tensors, 902 us: the
// norm 300 (5.4 TB/s), the second pass 638 alone (5.1 TB/s; a copy reaches 5.2).
// Read and stored through the caches as ordinary accesses do, the pass took 667
// and the call 976 (0.13e9 values in 121 tensors 131 us against 168).  Taking the
// values in the reverse order, the last read first, gained nothing.
#include "epilogue.h"
#include "grad_norm.h"

namespace gemmf32 {

namespace {

constexpr int kThreads = 256;

// A block's run of chunks, cut at the tensors' ends: use(tensor, first, count)
// for each piece.
template <typename F>
__device__ __forceinline__ void for_pieces(const GradTable& t, F&& use) {
    const int64_t total = t.first[t.count];
    int64_t c = total * blockIdx.x / gridDim.x;
    const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
    int lo = 0, hi = t.count - 1;                  // the tensor that holds chunk c
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    for (int i = lo; c < end; ++i) {
        const int64_t stop = t.first[i + 1] < end ? (int64_t)t.first[i + 1] : end;
        if (stop <= c) continue;                   // an empty tensor
        const int64_t from = (c - t.first[i]) * kGradChunk;
        const int64_t to = (stop - t.first[i]) * kGradChunk;
        use(i, from, (to < t.size[i] ? to : t.size[i]) - from);
        c = stop;
    }
}

// Values of p up to the next multiple of 16 bytes.
template <typename T>
__device__ __forceinline__ int64_t head_of(const T* p, int64_t n) {
    const int64_t h = (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / (int64_t)sizeof(T);
    return h < n ? h : n;
}

template <int TYPE>
__device__ __forceinline__ void add_squares(const void* base, int64_t from, int64_t n, double (&sum)[2]) {
    using T = typename Stored<TYPE>::T;
    constexpr int V = 16 / sizeof(T), U = 4;
    const T* p = static_cast<const T*>(base) + from;
    const int64_t head = head_of(p, n);
    auto one = [&](float v, int k) __attribute__((always_inline)) { sum[k & 1] = __builtin_fma((double)v, (double)v, sum[k & 1]); };
    if (threadIdx.x < head) one((float)p[threadIdx.x], 0);
    p += head;
    n -= head;
    const int64_t vectors = n / V;
    for (int64_t j = threadIdx.x; j < vectors; j += kThreads * U) {
        T v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * kThreads < vectors) __builtin_memcpy(v[u], p + (j + u * kThreads) * V, 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * kThreads < vectors) {
#pragma unroll
                for (int k = 0; k < V; ++k) one((float)v[u][k], k);
            }
    }
    const int64_t at = vectors * V + threadIdx.x;
    if (at < n) one((float)p[at], 1);
}

// The block's sum in thread 0's value: lanes in a tree, then the waves in order.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_down(v, d, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = part[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) s += part[w];
    return s;
}

__global__ __launch_bounds__(kThreads)
void grad_squares_kernel(GradTable t, double* partials) {
    double sum[2] = {0.0, 0.0};
    for_pieces(t, [&](int i, int64_t from, int64_t n) __attribute__((always_inline)) {
        if (t.type[i] == 0) add_squares<0>(t.in[i], from, n, sum);
        else if (t.type[i] == 1) add_squares<1>(t.in[i], from, n, sum);
        else add_squares<2>(t.in[i], from, n, sum);
    });
    const double s = block_sum(sum[0] + sum[1]);
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// The norm from the partials; the same in every thread and block.
__device__ __forceinline__ float norm_of(const double* partials, int count) {
    double s = 0.0;
    for (int i = threadIdx.x; i < count; i += kThreads) s += partials[i];
    return (float)__builtin_sqrt(block_sum(s));
}

__global__ __launch_bounds__(kThreads)
void grad_norm_kernel(const double* partials, int count, float* norm) {
    const float n = norm_of(partials, count);
    if (threadIdx.x == 0) *norm = n;
}

// 16 bytes that no one reads again soon.
typedef unsigned int Streamed __attribute__((ext_vector_type(4), aligned(2)));

template <int TYPE>
__device__ __forceinline__ void scale(const void* in, void* out, int64_t from, int64_t n, float factor) {
    using T = typename Stored<TYPE>::T;
    constexpr int V = 16 / sizeof(T), U = 4;
    const T* p = static_cast<const T*>(in) + from;
    T* q = static_cast<T*>(out) + from;
    const int64_t head = head_of(q, n);
    if (threadIdx.x < head) q[threadIdx.x] = (T)((float)p[threadIdx.x] * factor);
    p += head;
    q += head;
    n -= head;
    const int64_t vectors = n / V;
    for (int64_t j = threadIdx.x; j < vectors; j += kThreads * U) {
        T v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * kThreads < vectors) {
                const Streamed d = __builtin_nontemporal_load(reinterpret_cast<const Streamed*>(p + (j + u * kThreads) * V));
                __builtin_memcpy(v[u], &d, 16);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * kThreads < vectors) {
#pragma unroll
                for (int k = 0; k < V; ++k) v[u][k] = (T)((float)v[u][k] * factor);
                Streamed d;
                __builtin_memcpy(&d, v[u], 16);
                __builtin_nontemporal_store(d, reinterpret_cast<Streamed*>(q + (j + u * kThreads) * V));
            }
    }
    const int64_t at = vectors * V + threadIdx.x;
    if (at < n) q[at] = (T)((float)p[at] * factor);
}

// partials null: the norm is read from `norm`, else computed from the partials
// and written there by the first block of the only launch.
__global__ __launch_bounds__(kThreads)
void grad_clip_kernel(GradTable t, const double* partials, int count, float* norm, float max_norm, float eps) {
    float n;
    if (partials != nullptr) {
        n = norm_of(partials, count);
        if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    } else {
        n = *norm;
    }
    const double f = (double)max_norm / ((double)n + (double)eps);
    const float factor = f >= 1.0 ? 1.0f : (float)f;               // NaN stays NaN
    for_pieces(t, [&](int i, int64_t from, int64_t m) __attribute__((always_inline)) {
        if (factor == 1.0f && t.out[i] == t.in[i]) return;          // nothing changes
        if (t.type[i] == 0) scale<0>(t.in[i], t.out[i], from, m, factor);
        else if (t.type[i] == 1) scale<1>(t.in[i], t.out[i], from, m, factor);
        else scale<2>(t.in[i], t.out[i], from, m, factor);
    });
}

// The tensors from `from` on that a launch takes; returns the next one.
int64_t fill_table(const GradList& l, int64_t from, GradTable* t) {
    t->count = 0;
    t->first[0] = 0;
    int64_t i = from;
    for (; i < l.count && t->count < kGradTensors; ++i) {
        if (l.size[i] == 0) continue;
        const int64_t chunks = (l.size[i] + kGradChunk - 1) / kGradChunk;
        if (t->first[t->count] + chunks > 0xFFFFFFFFll) break;
        const int k = t->count++;
        t->in[k] = l.in[i];
        t->out[k] = l.out != nullptr ? l.out[i] : nullptr;
        t->size[k] = l.size[i];
        t->type[k] = (unsigned char)l.type[i];
        t->first[k + 1] = (uint32_t)(t->first[k] + chunks);
    }
    return i;
}

int blocks_of(const GradTable& t) { return (int)(t.first[t.count] < kGradBlocks ? t.first[t.count] : kGradBlocks); }

}  // namespace

int64_t grad_partials(int64_t count, const int64_t* size) {
    int64_t partials = 0, chunks = 0, taken = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (size[i] == 0) continue;
        const int64_t c = (size[i] + kGradChunk - 1) / kGradChunk;
        if (taken == kGradTensors || chunks + c > 0xFFFFFFFFll) {
            partials += chunks < kGradBlocks ? chunks : kGradBlocks;
            chunks = taken = 0;
        }
        chunks += c;
        ++taken;
    }
    return partials + (chunks < kGradBlocks ? chunks : kGradBlocks);
}

hipError_t launch_grad_squares(const GradList& l, double* partials, hipStream_t s) {
    GradTable t;
    for (int64_t i = 0; i < l.count;) {
        i = fill_table(l, i, &t);
        if (t.count == 0) break;
        const int blocks = blocks_of(t);
        hipLaunchKernelGGL(grad_squares_kernel, dim3(blocks), dim3(kThreads), 0, s, t, partials);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        partials += blocks;
    }
    return hipSuccess;
}

hipError_t launch_grad_norm(const double* partials, int64_t count, float* norm, hipStream_t s) {
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kThreads), 0, s, partials, (int)count, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const GradList& l, const double* partials, int64_t count, float* norm, float max_norm,
                            float eps, hipStream_t s) {
    GradTable t;
    for (int64_t i = 0; i < l.count;) {
        const int64_t next = fill_table(l, i, &t);
        if (t.count == 0) break;
        if (i == 0 && next < l.count && partials != nullptr) {
            const hipError_t err = launch_grad_norm(partials, count, norm, s);
            if (err != hipSuccess) return err;
            partials = nullptr;
        }
        i = next;
        hipLaunchKernelGGL(grad_clip_kernel, dim3(blocks_of(t)), dim3(kThreads), 0, s, t, partials, (int)count, norm,
                           max_norm, eps);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace gemmf32
