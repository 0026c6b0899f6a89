// mfma16_ksplit_core.h -- the K loop of the 16-bit product on 64 x 64 tiles
// whose four waves split the phases: one block's partial tiles, left in LDS
// (device code shared by mfma16_ksplit.hip, whose header explains the split
// and the LDS layouts, and by the kernels that end in another epilogue; not
// part of the public interface).
#pragma once

#include "mfma16_common.h"

namespace gemmf32 {

namespace {

template <bool KC>
struct KsplitTile16 {
    static constexpr int ELEMS = 64 * 32;               // per stage
    static constexpr int CPR = KC ? 4 : 8;               // 16-byte chunks per stored row
    static constexpr int RPC = 64 / CPR;                 // stored rows per 1 KB copy
    static constexpr int ROW = KC ? 32 : 64;             // elements per stored row
    static constexpr int READS = KC ? 4 : 8;             // LDS reads per step (4 fragments)
    static constexpr bool IS_KC = KC;
    __host__ __device__ static constexpr int swz(int r) {
        return KC ? (((r >> 3) & 1) << 1) : ((((r >> 1) & 1) << 1) | (((r >> 3) & 1) << 2));
    }
    // Copy j (0..3) fills stored rows RPC j .. RPC j + RPC - 1; lane l fills
    // physical chunk l % CPR of row RPC j + l / CPR, so it brings the logical
    // chunk (l % CPR) ^ swz(row).
    __host__ __device__ static int copy_row(int j, int lane) { return RPC * j + lane / CPR; }
    __host__ __device__ static int copy_chunk(int j, int lane) { return (lane % CPR) ^ swz(copy_row(j, lane)); }
    // k (relative to the phase) and first mn (relative to the tile) of the 8
    // values lane l of copy j brings.
    __host__ __device__ static int copy_k(int j, int lane) { return KC ? 8 * copy_chunk(j, lane) : copy_row(j, lane); }
    __host__ __device__ static int copy_mn(int j, int lane) { return KC ? copy_row(j, lane) : 8 * copy_chunk(j, lane); }
    // Byte offset of those 8 values from the stored matrix's base at k = 0.
    __host__ __device__ static int64_t copy_src(int j, int lane, int mn0, int64_t ld) {
        return KC ? 2 * ((int64_t)(mn0 + copy_row(j, lane)) * ld + copy_k(j, lane))
                  : 2 * ((int64_t)copy_row(j, lane) * ld + mn0 + copy_mn(j, lane));
    }
    __host__ __device__ static int64_t phase_bytes(int k0, int64_t ld) { return KC ? 2 * (int64_t)k0 : 2 * (int64_t)k0 * ld; }
    // Read base of lane l (bytes from stage 0 of this tile) for block f, and
    // the instruction offset of its read i (KC: i = 0; MC: i = 0, 1).
    //   KC: row 16 f + l % 16, chunk l / 16: 64 (l % 16) + 16 ((l / 16) ^ swz(l % 16)) + 1024 f
    //   MC: rows 8 (l / 16) + 4 i + (l % 16) / 4, values 16 f + 4 (l % 4) .. + 3
    __host__ __device__ static uint32_t read_base(int f, int lane) {
        const int j = lane & 15, g = lane >> 4;
        if constexpr (KC) {
            return (uint32_t)(64 * j + 16 * (g ^ swz(j)));
        } else {
            const int q = j >> 2, jj = j & 3;
            const int r0 = 8 * g + q;
            return (uint32_t)(128 * r0 + 16 * ((2 * f + (jj >> 1)) ^ swz(r0)) + 8 * (jj & 1));
        }
    }
    __host__ __device__ static constexpr uint32_t read_imm(int f, int i) { return KC ? 1024u * f : 512u * i; }
};

// The block's 64 x 64 tile at (m0, n0) of op(A) op(B), as four partial tiles
// in LDS, one per wave (256 threads), complete and visible to every wave on
// return.  TERMS, plane_a, plane_b: as for WideCore.
template <int FMT, bool KCA, bool KCB, int TERMS = 1>
struct KsplitCore {
    using TA = KsplitTile16<KCA>;
    using TB = KsplitTile16<KCB>;
    static constexpr int NS = 4, BK = 32;                       // stages per wave, k per phase
    static constexpr int STAGE = TA::ELEMS + TB::ELEMS;         // elements per stage (8 KB)
    static constexpr int WAVE_ELEMS = NS * STAGE;               // 32 KB per wave
    static constexpr int NREAD = TA::READS + TB::READS;
    static_assert(NREAD <= 16, "one read per matrix instruction at most");
    static constexpr int LDS_ELEMS = 4 * WAVE_ELEMS;

    __device__ static __forceinline__ void run(const Gemm16Args& p, int m0, int n0, uint16_t* lds,
                                               int64_t plane_a = 0, int64_t plane_b = 0) {
        const int tid = threadIdx.x;
        const int lane = tid & 63;
        const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

        // This wave's phases: local phase lp is phase 4 lp + w, at k0 = kof(lp).
        const int nph = TERMS * ceil_div(p.K, BK);
        // -24 .. 0 and a multiple of 8 with a k-contiguous factor (K is one then: a
        // lane's 8 values lie on one side of k = 0); -31 .. 0 with two mn-contiguous
        // ones, whose lanes bring one k each
        const int kbase = TERMS == 1 ? p.K - BK * nph : 0;
        const int P = nph > w ? (nph - 1 - w) / 4 + 1 : 0;
        auto kof = [&](int lp) __attribute__((always_inline)) { return kbase + BK * (4 * lp + w); };

        // Byte offset of the phase at k0 in each factor's planes (TERMS = 3: the K
        // loop runs over the pairs of planes one after the other).
        auto phase_a = [&](int k0) __attribute__((always_inline)) -> int64_t {
            if constexpr (TERMS == 1) return TA::phase_bytes(k0, p.lda);
            const int t = (k0 >= p.K) + (k0 >= 2 * p.K);
            return TA::phase_bytes(k0 - t * p.K, p.lda) + (t == 2 ? 2 * plane_a : 0);
        };
        auto phase_b = [&](int k0) __attribute__((always_inline)) -> int64_t {
            if constexpr (TERMS == 1) return TB::phase_bytes(k0, p.ldb);
            const int t = (k0 >= p.K) + (k0 >= 2 * p.K);
            return TB::phase_bytes(k0 - t * p.K, p.ldb) + (t == 1 ? 2 * plane_b : 0);
        };

        const int64_t a_rows = KCA ? p.M : p.K, a_cols = KCA ? p.K : p.M;
        const int64_t b_rows = KCB ? p.N : p.K, b_cols = KCB ? p.K : p.N;
        constexpr int kRawBufferWord3 = 0x00020000;
        constexpr uint32_t kPastEnd = 0x80000000u;           // beyond any descriptor here
        const __amdgpu_buffer_rsrc_t rsrc_a = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(p.A), (short)0, (int)(2 * (plane_a + (a_rows - 1) * p.lda + a_cols)), kRawBufferWord3);
        const __amdgpu_buffer_rsrc_t rsrc_b = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(p.B), (short)0, (int)(2 * (plane_b + (b_rows - 1) * p.ldb + b_cols)), kRawBufferWord3);
        // Copies 0..3 fill A's tile, 4..7 B's (byte offsets below 2^31: the
        // launcher checks the operands' extents).
        uint32_t doff[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            doff[j] = (uint32_t)TA::copy_src(j, lane, m0, p.lda);
            doff[4 + j] = (uint32_t)TB::copy_src(j, lane, n0, p.ldb);
            if (!KCA && m0 + TA::copy_mn(j, lane) >= a_cols) doff[j] = kPastEnd;
            if (!KCB && n0 + TB::copy_mn(j, lane) >= b_cols) doff[4 + j] = kPastEnd;
        }
        uint16_t* const wl = lds + w * WAVE_ELEMS;
        auto copy_at = [&](int j, uint32_t voff, int soff, int stage) __attribute__((always_inline)) {
            if (j < 4) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc_a, (__attribute__((address_space(3))) void*)(wl + stage * STAGE + 512 * j), 16, (int)voff, soff,
                    0, 0);
            } else {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc_b, (__attribute__((address_space(3))) void*)(wl + stage * STAGE + TA::ELEMS + 512 * (j - 4)), 16,
                    (int)voff, soff, 0, 0);
            }
        };
        // The wave's last phase (when it is not also its first) takes offsets of
        // its own with the phase folded in and a scalar offset of 0, so that the
        // chunk of an MC factor's last row across its last column meets the
        // descriptor's end by its per-lane offset.
        uint32_t dlast[8];
        {
            const int kl = kof(P > 0 ? P - 1 : 0);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t pb = j < 4 ? phase_a(kl) : phase_b(kl);
                dlast[j] = doff[j] == kPastEnd ? kPastEnd : (uint32_t)((int64_t)doff[j] + pb);
            }
        }
        // Copy j of local phase lp (k0 >= 0) into its stage; LAST: lp is the
        // wave's last phase.
        auto copy = [&](int j, int lp, int stage, auto lastc) __attribute__((always_inline)) {
            if constexpr (decltype(lastc)::value) {
                copy_at(j, dlast[j], 0, stage);
            } else {
                const int k0 = kof(lp);
                copy_at(j, doff[j], (int)(j < 4 ? phase_a(k0) : phase_b(k0)), stage);
            }
        };
        // The wave's first phase (k0 <= 0 only for phase 0), into stage 0: the
        // phase goes into each lane's offset, lanes below k = 0 point past the end.
        auto copy_first = [&]() __attribute__((always_inline)) {
            const int k0 = kof(0);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int kl = j < 4 ? TA::copy_k(j, lane) : TB::copy_k(j - 4, lane);
                const int64_t pb = j < 4 ? phase_a(k0) : phase_b(k0);
                copy_at(j, k0 + kl >= 0 && doff[j] != kPastEnd ? (uint32_t)((int64_t)doff[j] + pb) : kPastEnd, 0, 0);
            }
        };

        // Read bases (bytes, stage 0); the block and the stage are instruction offsets.
        const uint32_t wl0 = lds_addr(wl);
        uint32_t abase[KCA ? 1 : 4], bbase[KCB ? 1 : 4];
#pragma unroll
        for (int f = 0; f < (KCA ? 1 : 4); ++f) abase[f] = wl0 + TA::read_base(f, lane);
#pragma unroll
        for (int f = 0; f < (KCB ? 1 : 4); ++f) bbase[f] = wl0 + 2u * TA::ELEMS + TB::read_base(f, lane);

        u32x4 a[2][4], b[2][4];
        // Read i (0 .. NREAD - 1) of the phase in stage STG into set x: A's
        // fragments first (KC: read f = fragment f; MC: half i % 2 of fragment
        // i / 2), then B's.
        auto read_one = [&](auto tile, u32x4 (&x)[4], const uint32_t* base, auto stg, int i) __attribute__((always_inline)) {
            using T = decltype(tile);
            constexpr uint32_t SOFF = 2u * STAGE * decltype(stg)::value;
            if constexpr (T::IS_KC) {
                x[i] = lds_read128(base[0] + SOFF + T::read_imm(i, 0));
            } else {
                const int f = i / 2, r = i % 2;
                const u32x2 v = read_tr16_off(base[f], (int)(SOFF + T::read_imm(f, r)));
                x[f][2 * r] = v[0];
                x[f][2 * r + 1] = v[1];
            }
        };
        auto read_op = [&](auto stg, int t, int i) __attribute__((always_inline)) {
            if (i < TA::READS) read_one(TA{}, a[t], abase, stg, i);
            else read_one(TB{}, b[t], bbase, stg, i - TA::READS);
        };
        auto wait_set = [&](int t) __attribute__((always_inline)) {
            wait_tied(a[t]);
            wait_tied(b[t]);
        };

        floatx4 acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

        // One phase in stage U % NS, fragments in set U % 2 (U: the phase's
        // position in the unrolled group of NS): its 16 matrix instructions;
        // after instruction q (q < NREAD) read q of the next phase (from stage
        // (U + 1) % NS into the other set) if R, and after every odd one copy
        // q / 2 of local phase lp + 3 into stage (U + 3) % NS if C.
        auto phase = [&](auto uc, int lp, auto rc, auto cc, auto lastc) __attribute__((always_inline)) {
            constexpr int U = decltype(uc)::value;
            constexpr bool R = decltype(rc)::value, C = decltype(cc)::value;
            constexpr int T = U & 1;
            using NEXT = std::integral_constant<int, (U + 1) % NS>;
            unroll<16>([&](auto qc) __attribute__((always_inline)) {
                constexpr int q = decltype(qc)::value;
                acc[q / 4][q % 4] = mfma16x16<FMT>(a[T][q / 4], b[T][q % 4], acc[q / 4][q % 4]);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (R && q < NREAD) {
                    read_op(NEXT{}, T ^ 1, q);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if constexpr (C && q % 2 == 1) {
                    copy(q / 2, lp + 3, (U + 3) % NS, lastc);
                    __builtin_amdgcn_sched_barrier(0);
                }
            });
            if constexpr (R) wait_set(T ^ 1);
        };
        using yes = std::true_type;
        using no = std::false_type;

        if (P > 0) {
            copy_first();
#pragma unroll
            for (int lp = 1; lp < NS - 1; ++lp) {
                if (lp < P - 1) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) copy(j, lp, lp, no{});
                } else if (lp == P - 1) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) copy(j, lp, lp, yes{});
                }
            }
            // phase 0 has landed when at most the copies of phases 1 .. min(2, P - 1) are outstanding
            if (P >= 3) asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
            else if (P == 2) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
            else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
            for (int i = 0; i < NREAD; ++i) read_op(std::integral_constant<int, 0>{}, 0, i);
            wait_set(0);
            __builtin_amdgcn_sched_barrier(0);
            // Full phases in groups of NS (each copies the phase three ahead --
            // never the wave's last one -- and reads the next; the next phase's
            // copies have landed before its reads when at most those of phase
            // lp + 2 are outstanding), then the last ones.
            int lp0 = 0;
            for (; lp0 + NS + 3 < P; lp0 += NS) {
                unroll<NS>([&](auto uc) __attribute__((always_inline)) {
                    asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                    phase(uc, lp0 + decltype(uc)::value, yes{}, yes{}, no{});
                    __builtin_amdgcn_sched_barrier(0);
                });
            }
            for (; lp0 < P; lp0 += NS) {
                unroll<NS>([&](auto uc) __attribute__((always_inline)) {
                    const int lp = lp0 + decltype(uc)::value;
                    if (lp < P) {
                        if (lp + 2 < P) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
                        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                        __builtin_amdgcn_sched_barrier(0);
                        if (lp + 3 < P - 1) phase(uc, lp, yes{}, yes{}, no{});
                        else if (lp + 3 == P - 1) phase(uc, lp, yes{}, yes{}, yes{});
                        else if (lp + 1 < P) phase(uc, lp, yes{}, no{}, no{});
                        else phase(uc, lp, no{}, no{}, no{});
                        __builtin_amdgcn_sched_barrier(0);
                    }
                });
            }
        }

        // Partial tiles: register r of block (i, j) of lane l of wave v (row 16 i +
        // 4 (l / 16) + r, column 16 j + l % 16 of the tile) at float v 4096 +
        // ((4 i + j) 4 + r) 64 + l.
        __syncthreads();
        float* const part = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) part[w * 4096 + ((4 * i + j) * 4 + r) * 64 + lane] = acc[i][j][r];
        __syncthreads();
    }

    // Four consecutive columns of the finished tile (the partial tiles added
    // in wave order) for lane l of wave w, it = 0 .. 3: row 16 w + 4 ((l % 16)
    // / 4) + it, columns 16 (l / 16) + 4 (l % 4) .. + 3.  One 128-bit read per
    // partial tile, 16 lanes on 64 consecutive floats.
    __device__ static __forceinline__ int sum_row(int w, int lane, int it) { return 16 * w + 4 * ((lane & 15) >> 2) + it; }
    __device__ static __forceinline__ int sum_col(int lane) { return 16 * (lane >> 4) + 4 * (lane & 3); }
    __device__ static __forceinline__ floatx4 sum4(const uint16_t* lds, int w, int lane, int it) {
        const float* q = reinterpret_cast<const float*>(lds) + ((4 * w + (lane >> 4)) * 4 + it) * 64 + 4 * (lane & 15);
        floatx4 s = *reinterpret_cast<const floatx4*>(q);
#pragma unroll
        for (int v = 1; v < 4; ++v) s += *reinterpret_cast<const floatx4*>(q + 4096 * v);
        return s;
    }
};

}  // namespace

}  // namespace gemmf32
