// linear_w4.hip -- the product of a few rows with a weight held in 4 bits
// (a decoder's tokens), with the layer's epilogue.
//
//   Z[i][n] = sum over groups j of s[n][j] sum over k in j of
//             x[i][k] (q[n][k] - z[n][j]),     C = act(Z + bias) + residual
//
// The weight's bytes set the time, so it goes from memory straight into
// registers, and into matrix operands with one operation per value: q in the
// upper bits of a 16-bit float's fraction reads as 16 + q, exactly, and the 16
// is taken out together with the zero point,
//   sum x (q - z) = sum x (16 + q) - (16 + z) sum x,
// where sum x comes from one more matrix product, with ones, per 32 k: it lands
// in the registers where the rows' sums are.  The scale multiplies the group's
// binary32 sum: no weight is rounded.  (16 + q is at most four times |q - 8| on
// average, so the sums' rounding is 2 bits above an unshifted sum's: 2^-22.)
//
// A step is 128 k.  Lane (c = l % 16, g = l / 16) loads 16 bytes, 32 values,
// of column c from k 32 g on; a 4 x 4 transpose of dwords across the four lane
// groups (four lane swaps) then gives it, for each slice of 32 k, the eight
// values from 8 g on, as v_mfma_f32_16x16x32 takes them -- so that a matrix
// instruction stays inside one slice and so inside one scale group.  The pairs
// that a mask cuts out of a dword are values e and e + 4; x's eight values are
// put in that order (0 4 1 5 2 6 3 7).
//
// Waves of a block split K, each a run of whole steps, and add their sums in
// LDS in wave order.  Columns past N and rows past M repeat the last one and
// are not stored; values of x past K are zero, whatever the weight's bytes
// hold there.
#include "epilogue.h"
#include "linear_w4.h"
#include "mfma16_common.h"

namespace gemmf32 {

namespace {

constexpr int kStep = 128;

template <int FMT>
struct W4 {
    // 16 + q: the exponent of 16 and q below it
    static constexpr unsigned BASE = FMT == 0 ? 0x41804180u : 0x4C004C00u;
    static constexpr unsigned ONES = FMT == 0 ? 0x3F803F80u : 0x3C003C00u;
    static constexpr int SHIFT = FMT == 0 ? 3 : 6;        // q's place in the fraction
    __device__ static __forceinline__ u32x4 expand(unsigned w) {
        constexpr unsigned MASK = 0x000F000Fu << SHIFT;
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {                      // values i and i + 4
            const unsigned v = SHIFT >= 4 * i ? w << (SHIFT >= 4 * i ? SHIFT - 4 * i : 0)
                                              : w >> (SHIFT >= 4 * i ? 0 : 4 * i - SHIFT);
            r[i] = (v & MASK) | BASE;
        }
        return r;
    }
    // Eight values in the order 0 4 1 5 2 6 3 7.
    __device__ static __forceinline__ u32x4 reorder(u32x4 x) {
        return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                     __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
    }
    __device__ static __forceinline__ float value(unsigned bits) {
        if constexpr (FMT == 0) return __builtin_bit_cast(float, bits << 16);
        else return (float)__builtin_bit_cast(_Float16, (unsigned short)bits);
    }
};

// v[i] of lane group g <-> v[g] of lane group i (groups of 16 lanes).
__device__ __forceinline__ void transpose_groups(u32x4& v) {
    auto swap32 = [](unsigned a, unsigned b) { return __builtin_amdgcn_permlane32_swap(a, b, false, false); };
    auto swap16 = [](unsigned a, unsigned b) { return __builtin_amdgcn_permlane16_swap(a, b, false, false); };
    const auto p = swap32(v[0], v[2]), q = swap32(v[1], v[3]);
    const auto r = swap16(p[0], q[0]), s = swap16(p[1], q[1]);
    v = u32x4{r[0], r[1], s[0], s[1]};
}

// MT tiles of 16 rows, J of 16 columns, WAVES waves along K; SLICES: slices of
// 32 k per scale within a step (1, 2, or 4 for groups of 128 and more).
template <int FMT, int MT, int J, int WAVES, int SLICES>
__global__ __launch_bounds__(64 * WAVES)
void linear_w4_kernel(W4Args p, EpilogueArgs e) {
    constexpr int COLS = 16 * J, ROWS = 16 * MT, PITCH = COLS + 4, S = 4 / SLICES;
    __shared__ __attribute__((aligned(16))) float part[WAVES][ROWS][PITCH];
    using D = W4<FMT>;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n0 = COLS * (int)blockIdx.x, m0 = ROWS * (int)blockIdx.y;
    const int steps = ceil_div(p.K, kStep);
    const int begin = (int)((int64_t)steps * wave / WAVES), end = (int)((int64_t)steps * (wave + 1) / WAVES);
    const int bytes = (p.K + 1) / 2;

    const uint16_t* xrow[MT];
    const uint8_t* qrow[J];
    const uint16_t *srow[J], *zrow[J];
#pragma unroll
    for (int t = 0; t < MT; ++t) xrow[t] = p.X + (int64_t)min(m0 + 16 * t + c, p.M - 1) * p.ldx;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int64_t n = min(n0 + 16 * j + c, p.N - 1);
        qrow[j] = p.Q + n * p.ldq;
        srow[j] = p.scales + n * p.ld_scales;
        zrow[j] = p.zeros != nullptr ? p.zeros + n * p.ld_zeros : nullptr;
    }
    struct Step {
        u32x4 x[MT][4], q[J];
        unsigned s[J][(S + 1) / 2], z[J][(S + 1) / 2];      // two 16-bit values each
    };
    auto load_values = [](unsigned (&v)[(S + 1) / 2], const uint16_t* q) __attribute__((always_inline)) {
        if constexpr (S == 1) v[0] = q[0];
        else __builtin_memcpy(v, q, 2 * S);
    };
    auto load = [&](Step& st, int step) __attribute__((always_inline)) {
        const int k0 = step * kStep, at = k0 / 2 + 16 * g;
        const int group = k0 / p.group;
        if (k0 + kStep <= p.K) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                __builtin_memcpy(&st.q[j], qrow[j] + at, 16);
                load_values(st.s[j], srow[j] + group);
                if (p.zeros != nullptr) load_values(st.z[j], zrow[j] + group);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) __builtin_memcpy(&st.x[t][i], xrow[t] + k0 + 32 * i + 8 * g, 16);
        } else {                                            // the step across K
            const int groups = ceil_div(p.K, p.group);
#pragma unroll
            for (int j = 0; j < J; ++j) {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    unsigned v = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (at + 4 * d + b < bytes) v |= (unsigned)qrow[j][at + 4 * d + b] << (8 * b);
                    st.q[j][d] = v;
                }
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    const int at_group = min(group + i, groups - 1), place = 16 * (i % 2);
                    st.s[j][i / 2] = (i % 2 ? st.s[j][i / 2] : 0u) | (unsigned)srow[j][at_group] << place;
                    if (p.zeros != nullptr)
                        st.z[j][i / 2] = (i % 2 ? st.z[j][i / 2] : 0u) | (unsigned)zrow[j][at_group] << place;
                }
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = k0 + 32 * i + 8 * g;
                    u32x4 v = {0, 0, 0, 0};
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        if (k + b < p.K) v[b / 2] |= (unsigned)xrow[t][k + b] << (16 * (b % 2));
                    st.x[t][i] = v;
                }
        }
    };
    const floatx4 zero4 = {0.f, 0.f, 0.f, 0.f};
    const u32x4 ones = {D::ONES, D::ONES, D::ONES, D::ONES};
    floatx4 acc[MT][J];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < J; ++j) acc[t][j] = zero4;
    auto compute = [&](Step& st) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < J; ++j) transpose_groups(st.q[j]);
#pragma unroll
        for (int i = 0; i < S; ++i) {
            floatx4 sum[MT][J], sx[MT];
#pragma unroll
            for (int h = 0; h < SLICES; ++h) {
                const int slice = i * SLICES + h;
                u32x4 w[J];
#pragma unroll
                for (int j = 0; j < J; ++j) w[j] = D::expand(st.q[j][slice]);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const u32x4 x = D::reorder(st.x[t][slice]);
                    sx[t] = mfma16x16<FMT>(x, ones, h == 0 ? zero4 : sx[t]);
#pragma unroll
                    for (int j = 0; j < J; ++j) sum[t][j] = mfma16x16<FMT>(x, w[j], h == 0 ? zero4 : sum[t][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float s = D::value(st.s[j][i / 2] >> 16 * (i % 2));
                const float z = 16.0f + (p.zeros != nullptr ? D::value(st.z[j][i / 2] >> 16 * (i % 2)) : 8.0f);
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[t][j][r] = __builtin_fmaf(s, __builtin_fmaf(-z, sx[t][r], sum[t][j][r]), acc[t][j][r]);
            }
        }
    };
    if (begin < end) {
        Step s0, s1;
        load(s0, begin);
        for (int i = begin;;) {
            if (i + 1 < end) load(s1, i + 1);
            compute(s0);
            if (i + 1 >= end) break;
            if (i + 2 < end) load(s0, i + 2);
            compute(s1);
            if (i + 2 >= end) break;
            i += 2;
        }
    }
    // Register r of acc[t][j]: row 16 t + 4 g + r, column 16 j + c.
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) part[wave][16 * t + 4 * g + r][16 * j + c] = acc[t][j][r];
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * COLS / 4; i += 64 * WAVES) {
        const int row = i / (COLS / 4), tc = 4 * (i % (COLS / 4)), col = n0 + tc;
        if (m0 + row >= p.M || col >= p.N) continue;
        EpilogueRun<4, false> run;
        float bias[4];
        load_bias(e, col, bias);
        run.load(e, m0 + row, col);
        floatx4 s = *reinterpret_cast<const floatx4*>(&part[0][row][tc]);
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += *reinterpret_cast<const floatx4*>(&part[w][row][tc]);
        float v[4] = {s[0], s[1], s[2], s[3]};
        run.finish(e, m0 + row, col, bias, v);
    }
}

template <int FMT, int MT, int J, int WAVES>
void launch(const W4Args& p, const EpilogueArgs& e, hipStream_t s) {
    const dim3 grid(ceil_div(p.N, 16 * J), ceil_div(p.M, 16 * MT)), block(64 * WAVES);
    if (p.group == 32) hipLaunchKernelGGL((linear_w4_kernel<FMT, MT, J, WAVES, 1>), grid, block, 0, s, p, e);
    else if (p.group == 64) hipLaunchKernelGGL((linear_w4_kernel<FMT, MT, J, WAVES, 2>), grid, block, 0, s, p, e);
    else hipLaunchKernelGGL((linear_w4_kernel<FMT, MT, J, WAVES, 4>), grid, block, 0, s, p, e);
}

template <int FMT>
void launch_rows(const W4Args& p, const EpilogueArgs& e, hipStream_t s) {
    if (p.M <= 16) launch<FMT, 1, 1, 16>(p, e, s);
    else if (p.M <= 32) launch<FMT, 2, 2, 8>(p, e, s);
    else launch<FMT, 4, 2, 4>(p, e, s);
}

}  // namespace

hipError_t launch_linear_w4(const W4Args& p, const EpilogueArgs& e, hipStream_t s, int format) {
    if (format == 0) launch_rows<0>(p, e, s);
    else launch_rows<1>(p, e, s);
    return hipGetLastError();
}

}  // namespace gemmf32
