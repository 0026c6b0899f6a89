// mfma16_ksplit128_core.h -- the K loop of the 16-bit product on 128 x 128
// tiles whose four waves split the phases, and the exchange of their partial
// tiles (device code shared by mfma16_ksplit128.hip, whose header explains
// the split and the LDS layouts, and by the kernels that end in another
// epilogue; not part of the public interface).
#pragma once

#include "mfma16_common.h"

namespace gemmf32 {

namespace {

template <bool KC>
struct KsplitTile128 {
    static constexpr int ELEMS = 128 * 32;               // per stage
    static constexpr int BYTES = KC ? 8192 : 8 * 1056;   // per stage
    static constexpr int READS = KC ? 8 : 16;            // LDS reads per phase (8 fragments)
    static constexpr bool IS_KC = KC;
    // Copy j (0..7), lane l: the stored row (KC: mn; MC: k) and the logical
    // chunk of 8 values it brings, into LDS byte copy_dst(j) + 16 l.
    __host__ __device__ static int copy_row(int j, int lane) {
        if constexpr (KC) return 16 * j + lane / 4;
        const int pos = lane / 16;
        return 8 * (2 * (pos >> 1) + (j >> 2)) + 4 * (pos & 1) + (j & 3);
    }
    __host__ __device__ static int copy_chunk(int j, int lane) {
        return KC ? (lane % 4) ^ (((copy_row(j, lane) >> 3) & 1) << 1) : lane % 16;
    }
    __host__ __device__ static constexpr int copy_dst(int j) { return KC ? 1024 * j : 1056 * j; }
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
    // Read base of lane l (bytes from stage 0 of this tile) and the
    // instruction offset of read i of block f (KC: i = 0; MC: i = 0, 1).
    //   KC: row 16 f + l % 16, chunk l / 16
    //   MC: k row 8 (l / 16) + 4 i + (l % 16) / 4, values 16 f + 4 (l % 4) .. + 3
    __host__ __device__ static uint32_t read_base(int lane) {
        const int j = lane & 15, g = lane >> 4;
        if constexpr (KC) return (uint32_t)(64 * j + 16 * (g ^ (((j >> 3) & 1) << 1)));
        return (uint32_t)(1056 * ((j >> 2) + 4 * (g & 1)) + 512 * (g >> 1) + 8 * (j & 3));
    }
    __host__ __device__ static constexpr uint32_t read_imm(int f, int i) { return KC ? 1024u * f : 256u * i + 32u * f; }
};

// The block's 128 x 128 tile at (m0, n0) of op(A) op(B): run() leaves each
// wave's partial tile in its accumulators, exchange() adds them in wave
// order.  TERMS, plane_a, plane_b: as for WideCore.
template <int FMT, bool KCA, bool KCB, int TERMS = 1>
struct Ksplit128Core {
    using TA = KsplitTile128<KCA>;
    using TB = KsplitTile128<KCB>;
    static constexpr int BK = 32;                               // k per phase
    static constexpr int STAGE = TA::BYTES + TB::BYTES;         // bytes per stage (16 .. 16.5 KB)
    static constexpr int WAVE_BYTES = 2 * STAGE;                // two stages per wave
    static constexpr int PART_BYTES = 4 * 8 * 1024;             // a wave's outgoing partial blocks, per round
    static_assert(PART_BYTES <= WAVE_BYTES, "partials fit in the wave's stages");
    static constexpr int NREAD = TA::READS + TB::READS;         // 16 .. 32
    static constexpr int RO = 24;                               // instruction after which the first read goes
    static_assert(RO + NREAD <= 64, "a phase's reads fit in its instructions");
    static constexpr int LDS_BYTES = 4 * WAVE_BYTES;

    __device__ static __forceinline__ void run(const Gemm16Args& p, int m0, int n0, unsigned char* lds,
                                               floatx4 (&acc)[8][8], int64_t plane_a = 0, int64_t plane_b = 0) {
        const int tid = threadIdx.x;
        const int lane = tid & 63;
        const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

        // This wave's phases: local phase lp is phase 4 lp + w, at k0 = kof(lp).
        // It runs them at positions 0 .. P2 - 1: position 0 holds the last phase,
        // then (with an odd count, after a position that copies zeros) phases 0,
        // 1, .., P - 2; a wave with fewer than two phases runs two positions,
        // the missing ones copying zeros.  The phases that need per-lane offsets
        // -- the last and the first -- thus sit at positions 0 .. 2, copied in
        // the prologue and by the first two phases (peeled), and every copy in
        // the loop is the same.
        const int nph = TERMS * ceil_div(p.K, BK);
        // -24 .. 0 and a multiple of 8 with a k-contiguous factor (K is one then: a
        // lane's 8 values lie on one side of k = 0); -31 .. 0 with two mn-contiguous
        // ones, whose lanes bring one k each
        const int kbase = TERMS == 1 ? p.K - BK * nph : 0;
        const int P = nph > w ? (nph - 1 - w) / 4 + 1 : 0;
        const int odd = P & 1;
        const int P2 = P + odd < 2 ? 2 : P + odd;
        auto kof = [&](int lp) __attribute__((always_inline)) { return kbase + BK * (4 * lp + w); };
        auto phase_at = [&](int s) __attribute__((always_inline)) { return s == 0 ? P - 1 : s - 1 - odd; };

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
        // Copies 0..7 fill A's tile, 8..15 B's (byte offsets below 2^31: the
        // launcher checks the operands' extents).  Chunks of an MC factor wholly
        // past its last column point past the end in every phase.
        uint32_t doff[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            doff[j] = (uint32_t)TA::copy_src(j, lane, m0, p.lda);
            doff[8 + j] = (uint32_t)TB::copy_src(j, lane, n0, p.ldb);
            if (!KCA && m0 + TA::copy_mn(j, lane) >= a_cols) doff[j] = kPastEnd;
            if (!KCB && n0 + TB::copy_mn(j, lane) >= b_cols) doff[8 + j] = kPastEnd;
        }
        unsigned char* const wl = lds + w * WAVE_BYTES;
        auto copy_at = [&](int j, uint32_t voff, int soff, int stage) __attribute__((always_inline)) {
            if (j < 8) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc_a, (__attribute__((address_space(3))) void*)(wl + stage * STAGE + TA::copy_dst(j)), 16,
                    (int)voff, soff, 0, 0);
            } else {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc_b, (__attribute__((address_space(3))) void*)(wl + stage * STAGE + TA::BYTES + TB::copy_dst(j - 8)),
                    16, (int)voff, soff, 0, 0);
            }
        };
        // Copy j of the phase at position s >= 4 (phase s - 1 - odd >= 2, the
        // phase in the scalar offset) into `stage`; positions from P2 on copy
        // into stages nothing reads afterwards (the phase past the last one as
        // the wave's second, so that nothing past the factors is read).
        auto copy = [&](int j, int s, int stage) __attribute__((always_inline)) {
            const int lp = s - 1 - odd;
            const int k0 = kof(lp < P ? lp : 1);
            copy_at(j, doff[j], (int)(j < 8 ? phase_a(k0) : phase_b(k0)), stage);
        };
        // Copy j of the phase at position s with the phase in each lane's offset
        // (scalar offset 0) into `stage`: lanes below k = 0 or at k >= K, chunks
        // past an MC factor's last column, and positions holding no phase point
        // past the end.
        auto copy_folded = [&](int j, int s, int stage) __attribute__((always_inline)) {
            const int lp = phase_at(s);
            const int k0 = kof(lp);
            const int kl = j < 8 ? TA::copy_k(j, lane) : TB::copy_k(j - 8, lane);
            const int64_t pb = j < 8 ? phase_a(k0) : phase_b(k0);
            const bool inside = lp >= 0 && lp < P && k0 + kl >= 0 && k0 + kl < TERMS * p.K && doff[j] != kPastEnd;
            copy_at(j, inside ? (uint32_t)((int64_t)doff[j] + pb) : kPastEnd, 0, stage);
        };

        // Read bases (bytes, stage 0); block, read and stage are instruction offsets.
        const uint32_t abase = lds_addr(wl) + TA::read_base(lane);
        const uint32_t bbase = lds_addr(wl) + (uint32_t)TA::BYTES + TB::read_base(lane);

        // Fragments, two sets: a KC factor's as 128-bit values (one read each),
        // an MC factor's as the two 64-bit halves its two reads bring, put
        // together only as the matrix instruction's operand.
        u32x4 aq[2][8], bq[2][8];
        u32x2 ah[2][8][2], bh[2][8][2];
        // Read i (0 .. READS - 1) of one factor's fragments of the phase in stage
        // STG into set (q, h): KC, fragment i; MC, half i % 2 of fragment i / 2.
        auto read_one = [&](auto tile, u32x4 (&q)[8], u32x2 (&hv)[8][2], uint32_t base, auto stg, int i)
                            __attribute__((always_inline)) {
            using T = decltype(tile);
            constexpr uint32_t SOFF = (uint32_t)STAGE * decltype(stg)::value;
            if constexpr (T::IS_KC) q[i] = lds_read128(base + SOFF + T::read_imm(i, 0));
            else hv[i / 2][i % 2] = read_tr16_off(base, (int)(SOFF + T::read_imm(i / 2, i % 2)));
        };
        auto read_op = [&](auto stg, int t, int i) __attribute__((always_inline)) {
            if (i < TA::READS) read_one(TA{}, aq[t], ah[t], abase, stg, i);
            else read_one(TB{}, bq[t], bh[t], bbase, stg, i - TA::READS);
        };
        auto frag_a = [&](int t, int i) __attribute__((always_inline)) -> u32x4 {
            if constexpr (KCA) return aq[t][i];
            else return u32x4{ah[t][i][0][0], ah[t][i][0][1], ah[t][i][1][0], ah[t][i][1][1]};
        };
        auto frag_b = [&](int t, int j) __attribute__((always_inline)) -> u32x4 {
            if constexpr (KCB) return bq[t][j];
            else return u32x4{bh[t][j][0][0], bh[t][j][0][1], bh[t][j][1][0], bh[t][j][1][1]};
        };
        auto wait_set = [&](int t) __attribute__((always_inline)) {
            if constexpr (KCA) wait_tied(aq[t]);
            else wait_tied(ah[t]);
            if constexpr (KCB) wait_tied(bq[t]);
            else wait_tied(bh[t]);
        };

#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

        // The phase at position lp in stage U = lp % 2, its fragments in set U:
        // the 64 matrix instructions; after odd instruction q < 32, copy q / 2 of
        // position lp + 2 into stage U (FOLDED: with per-lane offsets); after
        // instruction RO - 1, wait until only this phase's 12 copies so far may
        // be in flight (those of position lp + 1 have landed, in order); after
        // instruction q >= RO, read q - RO of position lp + 1 from stage U ^ 1
        // into set U ^ 1.
        auto phase = [&](auto uc, int lp, auto foldc) __attribute__((always_inline)) {
            constexpr int U = decltype(uc)::value;
            using NEXT = std::integral_constant<int, U ^ 1>;
            unroll<64>([&](auto qc) __attribute__((always_inline)) {
                constexpr int q = decltype(qc)::value;
                acc[q / 8][q % 8] = mfma16x16<FMT>(frag_a(U, q / 8), frag_b(U, q % 8), acc[q / 8][q % 8]);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (q % 2 == 1 && q < 32) {
                    if constexpr (decltype(foldc)::value) copy_folded(q / 2, lp + 2, U);
                    else copy(q / 2, lp + 2, U);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if constexpr (q == RO - 1) {
                    asm volatile("s_waitcnt vmcnt(12)" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                }
                if constexpr (q >= RO && q < RO + NREAD) {
                    read_op(NEXT{}, U ^ 1, q - RO);
                    __builtin_amdgcn_sched_barrier(0);
                }
            });
            wait_set(U ^ 1);
        };
        using s0 = std::integral_constant<int, 0>;
        using s1 = std::integral_constant<int, 1>;

#pragma unroll
        for (int j = 0; j < 16; ++j) copy_folded(j, 0, 0);
#pragma unroll
        for (int j = 0; j < 16; ++j) copy_folded(j, 1, 1);
        asm volatile("s_waitcnt vmcnt(16)" ::: "memory");                  // position 0 has landed
#pragma unroll
        for (int i = 0; i < NREAD; ++i) read_op(s0{}, 0, i);
        wait_set(0);
        __builtin_amdgcn_sched_barrier(0);
        phase(s0{}, 0, std::true_type{});
        __builtin_amdgcn_sched_barrier(0);
        phase(s1{}, 1, std::true_type{});
        __builtin_amdgcn_sched_barrier(0);
        for (int pos = 2; pos < P2; pos += 2) {
            phase(s0{}, pos, std::false_type{});
            __builtin_amdgcn_sched_barrier(0);
            phase(s1{}, pos + 1, std::false_type{});
            __builtin_amdgcn_sched_barrier(0);
        }
        // the copies aimed past the last position land in this wave's stages
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    // Partial tiles, in two rounds.  In round a, wave v adds block row
    // 4 a + v of the tile (16 rows) over the four waves, in wave order.  Each
    // wave writes its four block rows of the round into its own stages (no
    // copy in flight and no read pending, and no other wave reads them before
    // the barrier), block row 4 a + v at float 2048 v, each as 16 rows of 128 floats, row-major, the 16-float segments of row rho
    // XORed by 16 ((rho / 4) mod 2): register r of block (i, j) of lane l
    // (row 4 (l / 16) + r, column 16 j + l % 16) is one 32-bit write per
    // (j, r), conflict free at 32 lanes a cycle.  Wave v then reads, for
    // it = 0..7, row 2 it + l / 32, columns 4 (l % 32) .. + 3 of its block
    // row from each wave -- one 128-bit read, conflict free under the
    // measured grouping -- and adds them: use(a, it, row, column, sum, slot),
    // row and column in the tile, 32 lanes on one row; `slot` is where the
    // sum's first addend lay, which no other wave reads.  done(a) follows the
    // round's last use.  (Taking the block rows in order keeps the allocator
    // from moving accumulators inside the phase loop.)
    // (rho / 4) mod 2 is (l / 16) mod 2 for a write and (it / 2) mod 2 for a
    // read, so two per-lane bases each serve every address (instruction
    // offsets): writes of even and of odd j; reads without and with the XOR.
    template <typename F, typename G>
    __device__ static __forceinline__ void exchange(const floatx4 (&acc)[8][8], unsigned char* lds, F&& use, G&& done) {
        const int lane = threadIdx.x & 63;
        const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        unsigned char* const wl = lds + w * WAVE_BYTES;
        const int b16 = (lane >> 4) & 1;
        float* const wbase_even = reinterpret_cast<float*>(wl) + 512 * (lane >> 4) + (lane & 15) + 16 * b16;
        float* const wbase_odd = reinterpret_cast<float*>(wl) + 512 * (lane >> 4) + (lane & 15) - 16 * b16;
        const int colq = 4 * (lane & 31);
        const float* const rbase0 = reinterpret_cast<const float*>(lds) + 2048 * w + 128 * (lane >> 5) + colq;
        const float* const rbase1 = reinterpret_cast<const float*>(lds) + 2048 * w + 128 * (lane >> 5) + (colq ^ 16);
        unroll<2>([&](auto ac) __attribute__((always_inline)) {
            constexpr int a = decltype(ac)::value;
            if constexpr (a == 1) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // round 0 is read
            unroll<4>([&](auto vc) __attribute__((always_inline)) {
                constexpr int v = decltype(vc)::value;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        ((j & 1) ? wbase_odd : wbase_even)[2048 * v + 128 * r + 16 * j] = acc[4 * a + v][j][r];
            });
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int rho = 2 * it + (lane >> 5);
                const float* const rb = ((it >> 1) & 1) ? rbase1 : rbase0;
                floatx4 sum = *reinterpret_cast<const floatx4*>(rb + 256 * it);
#pragma unroll
                for (int u = 1; u < 4; ++u) sum += *reinterpret_cast<const floatx4*>(rb + (WAVE_BYTES / 4) * u + 256 * it);
                use(a, it, 16 * (4 * a + w) + rho, colq, sum, const_cast<float*>(rb) + 256 * it);
            }
            done(a);
        });
    }
};

}  // namespace

}  // namespace gemmf32
