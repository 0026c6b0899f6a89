// epilogue.h -- what happens to an entry of a product before it is stored:
// bias, activation and residual of a fully connected layer, or the
// activation's derivative of its backward pass (device code shared by the
// kernels that end in it; not part of the public interface).
//
//   forward    z = v + bias[col];      C = act(z) + residual;  z kept if asked
//   gradient   d = (v + residual) act'(z);  C = d;  column sums of d if asked
//
// v, z, d and the column sums are binary32; C, residual, bias and the kept z
// are 16-bit or binary32 values, each rounded once, when it is stored (the
// column sums add d before its rounding).
#pragma once

#include "launch.h"

#include <type_traits>

namespace gemmf32 {

namespace {

// Types of stored values: 0 bfloat16, 1 binary16, 2 binary32.
template <int TYPE>
struct Stored;
template <>
struct Stored<0> {
    using T = __bf16;
};
template <>
struct Stored<1> {
    using T = _Float16;
};
template <>
struct Stored<2> {
    using T = float;
};

// W consecutive stored values as binary32, and back (nearest-even), the first
// `valid` of them (the rest read as 0 and are not written).  The values need
// their own alignment only; gfx9 runs global memory in unaligned mode, so the
// compiler may use one wide access.
template <int TYPE, int W>
__device__ __forceinline__ void load_values(const void* base, int64_t index, int valid, float (&v)[W]) {
    using T = typename Stored<TYPE>::T;
    const T* p = static_cast<const T*>(base) + index;
    if (valid >= W) {
        T raw[W];
        __builtin_memcpy(raw, p, sizeof(raw));
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = (float)raw[e];
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = e < valid ? (float)p[e] : 0.0f;
    }
}
template <int TYPE, int W>
__device__ __forceinline__ void store_values(void* base, int64_t index, int valid, const float (&v)[W]) {
    using T = typename Stored<TYPE>::T;
    T* p = static_cast<T*>(base) + index;
    if (valid >= W) {
        T raw[W];
#pragma unroll
        for (int e = 0; e < W; ++e) raw[e] = (T)v[e];
        __builtin_memcpy(p, raw, sizeof(raw));
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e < valid) p[e] = (T)v[e];
    }
}
template <int W>
__device__ __forceinline__ void load_values(int type, const void* base, int64_t index, int valid, float (&v)[W]) {
    if (type == 0) load_values<0>(base, index, valid, v);
    else if (type == 1) load_values<1>(base, index, valid, v);
    else load_values<2>(base, index, valid, v);
}
template <int W>
__device__ __forceinline__ void store_values(int type, void* base, int64_t index, int valid, const float (&v)[W]) {
    if (type == 0) store_values<0>(base, index, valid, v);
    else if (type == 1) store_values<1>(base, index, valid, v);
    else store_values<2>(base, index, valid, v);
}

// e^x and 1 / x on the hardware's 1-ulp units: with the argument's scaling
// by log2 e (rounded, and a rounding of the product), e^x is within
// (2 + 1.23 |x|) 2^-24 of its value.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// The normal distribution function Phi(z) and its density's exponential
// e^(-z^2 / 2).  With t = 1 / (1 + 0.28 |z|), e^(z^2 / 2) Phi(-|z|) is t
// times a polynomial in t: eighth degree, fitted to half the scaled
// complementary error function in binary64 for the smallest largest relative
// error; evaluated in binary32 5.1e-7, and 7e-7 where the reciprocal is a unit
// in the last place off.  Phi(z) = 1 - Phi(-z) for z > 0, so
// small tails keep their relative accuracy.
__device__ __forceinline__ float normal_cdf(float z, float* density) {
    const float a = __builtin_fabsf(z);
    const float t = fast_rcp(1.0f + 0.28f * a);
    float q = 0.02475812f;
    q = __builtin_fmaf(q, t, -0.09374318f);
    q = __builtin_fmaf(q, t, 0.09266892f);
    q = __builtin_fmaf(q, t, -0.00665205f);
    q = __builtin_fmaf(q, t, 0.07287117f);
    q = __builtin_fmaf(q, t, 0.0836053f);
    q = __builtin_fmaf(q, t, 0.10308819f);
    q = __builtin_fmaf(q, t, 0.11169959f);
    q = __builtin_fmaf(q, t, 0.11170386f);
    const float g = fast_exp(-0.5f * z * z);
    const float tail = g * (t * q);
    *density = g;
    return z > 0.0f ? 1.0f - tail : tail;
}

// Activations (GEMM_ACT_*) and their derivatives.  NaN stays NaN; infinities
// give the limits (0 and +inf, derivatives 0 and 1): a pre-activation past
// binary16's range is kept as one.  So the factor z, which would meet a zero
// there, is held at a finite value where the other factor is zero already.
//   gelu_tanh: (1 + tanh u) / 2 = 1 / (1 + e^(-2 u)), u = c (z + 0.044715 z^3),
//   c = sqrt(2 / pi).
enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
constexpr float kTanhC = 0.79788456080286536f, kTanhCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float activate_one(float z) {
    const float finite = __builtin_fmaxf(z, -3.4028234663852886e38f);   // NaN is in the other factor
    if constexpr (ACT == kActRelu) return z <= 0.0f ? 0.0f : z;
    if constexpr (ACT == kActGelu) {
        float g;
        return finite * normal_cdf(z, &g);
    }
    if constexpr (ACT == kActGeluTanh) {
        const float u2 = -2.0f * kTanhC * z * __builtin_fmaf(kTanhCubic * z, z, 1.0f);
        return finite * fast_rcp(1.0f + fast_exp(u2));
    }
    if constexpr (ACT == kActSilu) return finite * fast_rcp(1.0f + fast_exp(-z));
    return z;
}

template <int ACT>
__device__ __forceinline__ float activate_derivative_one(float z) {
    if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == kActGelu) {
        float g;
        const float cdf = normal_cdf(z, &g);
        const float near = __builtin_fabsf(z) > 30.0f ? 30.0f : z;      // g is 0 past 30
        return __builtin_fmaf(near * 0.39894228040143268f, g, cdf);
    }
    if constexpr (ACT == kActGeluTanh) {
        const float u2 = -2.0f * kTanhC * z * __builtin_fmaf(kTanhCubic * z, z, 1.0f);
        const float s = fast_rcp(1.0f + fast_exp(u2));
        // d u2 / dz = -2 c (1 + 3 0.044715 z^2); s' = -s (1 - s) du2.  Past 30, s
        // is 0 or 1 and s (1 - s) is 0.
        const float near = __builtin_fabsf(z) > 30.0f ? 30.0f : z;
        const float du = 2.0f * kTanhC * __builtin_fmaf(3.0f * kTanhCubic * near, near, 1.0f);
        return __builtin_fmaf(near, du * (s * (1.0f - s)), s);
    }
    if constexpr (ACT == kActSilu) {
        const float s = fast_rcp(1.0f + fast_exp(-z));
        const float near = __builtin_fabsf(z) > 100.0f ? 100.0f : z;    // s is 0 or 1 past 100
        return __builtin_fmaf(near, s * (1.0f - s), s);
    }
    return 1.0f;
}

// v = act(v), or v *= act'(z): one branch for the run, not one per value.
template <int W>
__device__ __forceinline__ void activate(int act, float (&v)[W]) {
    auto each = [&](auto a) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = activate_one<decltype(a)::value>(v[i]);
    };
    if (act == kActRelu) each(std::integral_constant<int, kActRelu>{});
    else if (act == kActGelu) each(std::integral_constant<int, kActGelu>{});
    else if (act == kActGeluTanh) each(std::integral_constant<int, kActGeluTanh>{});
    else if (act == kActSilu) each(std::integral_constant<int, kActSilu>{});
}
template <int W>
__device__ __forceinline__ void times_derivative(int act, const float (&z)[W], float (&v)[W]) {
    auto each = [&](auto a) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] *= activate_derivative_one<decltype(a)::value>(z[i]);
    };
    if (act == kActRelu) each(std::integral_constant<int, kActRelu>{});
    else if (act == kActGelu) each(std::integral_constant<int, kActGelu>{});
    else if (act == kActGeluTanh) each(std::integral_constant<int, kActGeluTanh>{});
    else if (act == kActSilu) each(std::integral_constant<int, kActSilu>{});
}

// W stored values as loaded, of a type known at run time only.
template <int W>
struct RawRun {
    unsigned w[W];
    __device__ __forceinline__ void load(int type, const void* base, int64_t index, int valid) {
        if (type == 2) {
            const float* p = static_cast<const float*>(base) + index;
            if (valid >= W) {
                __builtin_memcpy(w, p, 4 * W);
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) w[e] = e < valid ? __builtin_bit_cast(unsigned, p[e]) : 0u;
            }
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(base) + index;
            if (valid >= W) {
                __builtin_memcpy(w, p, 2 * W);
            } else {
#pragma unroll
                for (int e = 0; e < W / 2; ++e)
                    w[e] = (2 * e < valid ? (unsigned)p[2 * e] : 0u) |
                           (2 * e + 1 < valid ? (unsigned)p[2 * e + 1] << 16 : 0u);
            }
        }
    }
    __device__ __forceinline__ void values(int type, float (&v)[W]) const {
        if (type == 2) {
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = __builtin_bit_cast(float, w[e]);
        } else if (type == 0) {
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                v[2 * e] = __builtin_bit_cast(float, w[e] << 16);
                v[2 * e + 1] = __builtin_bit_cast(float, w[e] & 0xFFFF0000u);
            }
        } else {
            _Float16 h[W];
            __builtin_memcpy(h, w, 2 * W);
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = (float)h[e];
        }
    }
};

// W consecutive columns from `col` of a row inside C (columns past N are
// skipped): what the epilogue reads there, loaded ahead of its use, and the
// epilogue.  GRADIENT: the mode, EpilogueArgs::gradient.
template <int W, bool GRADIENT>
struct EpilogueRun {
    RawRun<W> residual;
    unsigned preact[GRADIENT ? W / 2 : 1];
    __device__ __forceinline__ void load(const EpilogueArgs& e, int row, int col) {
        if (e.residual != nullptr) residual.load(e.c_type, e.residual, (int64_t)row * e.ldr + col, e.N - col);
        if constexpr (GRADIENT) {
            if (e.act != kActNone) {
                RawRun<W> z;
                z.load(e.z_type, e.preact, (int64_t)row * e.ldz + col, e.N - col);
#pragma unroll
                for (int i = 0; i < W / 2; ++i) preact[i] = z.w[i];
            }
        }
    }
    // v: the product's entries on entry; d on return in gradient mode (0 past
    // N).  bias: the columns' (forward mode; zeros without one).
    __device__ __forceinline__ void finish(const EpilogueArgs& e, int row, int col, const float (&bias)[W],
                                           float (&v)[W]) const {
        const int valid = e.N - col;
        apply(
            e, bias, v,
            [&](const float (&z)[W]) __attribute__((always_inline)) {
                store_values(e.z_type, e.preact, (int64_t)row * e.ldz + col, valid, z);
            },
            [&](const float (&c)[W]) __attribute__((always_inline)) {
                store_values(e.c_type, e.C, (int64_t)row * e.ldc + col, valid, c);
            });
        if constexpr (GRADIENT) {
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = i < valid ? v[i] : 0.0f;
        }
    }
    // The epilogue of whole runs at given places: C's at c_base + c_at
    // elements, the kept pre-activation's at z_base + z_at.
    __device__ __forceinline__ void finish_at(const EpilogueArgs& e, char* c_base, uint32_t c_at, char* z_base,
                                              uint32_t z_at, const float (&bias)[W], float (&v)[W]) const {
        apply(
            e, bias, v,
            [&](const float (&z)[W]) __attribute__((always_inline)) {
                if (e.z_type == 0) store_whole<0>(z_base, 2 * z_at, z);
                else store_whole<1>(z_base, 2 * z_at, z);
            },
            [&](const float (&c)[W]) __attribute__((always_inline)) {
                if (e.c_type == 0) store_whole<0>(c_base, 2 * c_at, c);
                else if (e.c_type == 1) store_whole<1>(c_base, 2 * c_at, c);
                else store_whole<2>(c_base, 4 * c_at, c);
            });
    }
    template <int TYPE>
    __device__ static __forceinline__ void store_whole(char* base, uint32_t byte, const float (&v)[W]) {
        typename Stored<TYPE>::T raw[W];
#pragma unroll
        for (int i = 0; i < W; ++i) raw[i] = (typename Stored<TYPE>::T)v[i];
        __builtin_memcpy(base + byte, raw, sizeof(raw));
    }
    template <typename SZ, typename SC>
    __device__ __forceinline__ void apply(const EpilogueArgs& e, const float (&bias)[W], float (&v)[W], SZ&& store_z,
                                          SC&& store_c) const {
        float r[W];
        if (e.residual != nullptr) residual.values(e.c_type, r);
        if constexpr (GRADIENT) {
            if (e.residual != nullptr) {
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] += r[i];
            }
            if (e.act != kActNone) {
                RawRun<W> raw;
                float z[W];
#pragma unroll
                for (int i = 0; i < W / 2; ++i) raw.w[i] = preact[i];
                raw.values(e.z_type, z);
                times_derivative(e.act, z, v);
            }
            if (e.C != nullptr) store_c(v);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] += bias[i];
            if (e.preact != nullptr) store_z(v);
            activate(e.act, v);
            if (e.residual != nullptr) {
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] += r[i];
            }
            store_c(v);
        }
    }
};

// The bias of W columns from `col` (zeros without one).
template <int W>
__device__ __forceinline__ void load_bias(const EpilogueArgs& e, int col, float (&b)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) b[i] = 0.0f;
    if (e.bias != nullptr && col < e.N) load_values(e.bias_type, e.bias, col, e.N - col, b);
}

}  // namespace

}  // namespace gemmf32
