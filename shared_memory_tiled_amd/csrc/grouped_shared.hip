// grouped_shared.hip -- the grouped layer on tiles that share a CU with other
// blocks: 128 x 256 and 128 x 128, 64 x 256 and 64 x 128 (GroupedSharedCore).
//
// The scheduled tiles own a CU: their start (the first copies' latency) and
// their epilogue (12 to 20 us) pass with the matrix units idle, which is the
// most of a tile's time where K is short -- a weight's gradient over an expert's
// few hundred rows above all -- and groups of unequal rows leave their last
// round badly filled.  Here two or three blocks share a CU's LDS and registers (of
// the 64 x 128 tiles through registers four), so that one computes while another
// starts or stores.
//
// K goes in phases of 32 through a ring of LDS stages: while one is computed the
// copies of the next are in flight, about 96 KB on a CU whatever the tile, which
// is what the memory's latency takes.  Per phase a wave issues its share of the
// 1 KB copies straight into LDS and its matrix instructions, and passes one
// barrier.  Problems that the copies do not take (DIRECT false: odd widths,
// leading dimensions or bases, an odd K, operands past 2 GiB) go
// through registers instead: runs of 8 values loaded wherever they lie, three
// phases ahead, then written to the same places of one of two stages.  The stages
// have the layouts of the 128-wide k-split tiles
// (KsplitTile128): one for A's 128 rows or half of one for 64, one or two side
// by side for B's columns.
//
// Measured: 16384 x 4096 x 4096 bf16 over 8 groups 542 to 563 us (1.0 PFLOP/s, the
// matrix units 54 % busy at the clock that their power allows; its tiles are 4 to
// 4.4 rounds), 4096 x 1024 x 2048 over 64 65 (the weights' read, 4.7 TB/s), 16 x 2048
// x 4096 over 16 28.5 and the pass over four shares of K 4 (6 TB/s); gradients
// (alone): 16384 x 4096 x 4096 over 8 470 to 480, 8192 x 2048 x 4096 over 16 147 to
// 150, 4096 x 1024 x 2048 over 64 59.
#include "epilogue.h"
#include "grouped_kernels.h"
#include "mfma16_ksplit128_core.h"
#include "staged_tile.h"

namespace gemmf32 {

namespace {

// Zeros over the block's BM x BN tile at (m0, n0): the gradient of a weight
// that no row chose.
template <int BM, int BN>
__device__ __forceinline__ void zero_tile(const EpilogueArgs& e, int m0, int n0) {
    const float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = threadIdx.x; i < BM * BN / 8; i += 256) {
        const int row = m0 + i / (BN / 8), col = n0 + 8 * (i % (BN / 8));
        if (row < e.M && col < e.N) store_values(e.c_type, e.C, (int64_t)row * e.ldc + col, e.N - col, v);
    }
}

// Waits until at most N of this wave's copies are in flight and its LDS reads are
// done.
template <int N>
__device__ __forceinline__ void wait_ring() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// The same for `ahead` phases of C copies each beyond the one waited for, at
// most N of them in flight.
template <int N, int C>
__device__ __forceinline__ void wait_phase(int ahead) {
    if (N == 0 || ahead >= N) wait_ring<N * C>();
    else wait_phase<(N > 0 ? N - 1 : 0), C>(ahead);
}

// 16 bytes at any address that a 16-bit value may have, past the caches: what
// no one reads soon need not push out what the other blocks read.
__device__ __forceinline__ void store_streamed(char* p, u32x4 v) {
    typedef u32x4 Bytes __attribute__((aligned(2)));
    __builtin_nontemporal_store(v, reinterpret_cast<Bytes*>(p));
}

// BM rows (64 only with A k-contiguous) x 128 NB columns, BLOCKS to a CU.
template <int FMT, bool KCA, bool KCB, int BM_, int NB, int STAGES, int BLOCKS, bool DIRECT>
struct GroupedSharedCore {
    using TA = KsplitTile128<KCA>;
    using TB = KsplitTile128<KCB>;
    static constexpr int BM = BM_, BN = 128 * NB, BK = 32;
    static_assert(BM == 128 || (BM == 64 && KCA), "tile");
    // 64 x 256: four waves side by side; else two by two
    static constexpr int WROWS = BM == 64 && NB == 2 ? 1 : 2, WCOLS = 4 / WROWS;
    static constexpr int FM = BM / 16 / WROWS, FN = BN / 16 / WCOLS;
    static constexpr int A_BYTES = TA::BYTES * BM / 128, STAGE = A_BYTES + NB * TB::BYTES;
    static constexpr int CA = BM / 64, CB = 2 * NB, COPIES = CA + CB;            // per wave and phase
    using Staged = StagedTile<FM, FN>;
    using Run = EpilogueRun<8, false>;
    static constexpr int PATCHES = 4 * Staged::PATCH * 4;
    static constexpr int BIAS = STAGES * STAGE > PATCHES ? STAGES * STAGE : PATCHES;   // its place in LDS
    static constexpr int LDS_BYTES = BIAS + 4 * BN;
    static_assert(BLOCKS * LDS_BYTES <= 163840, "blocks to a CU");

    // Where a wave reads its fragments in stage 0: its FM blocks of 16 rows and FN
    // of 16 columns (of one half, which holds 8 of them).
    struct Fragments {
        uint32_t a_at, b_at;
        __device__ __forceinline__ Fragments(const unsigned char* lds, int lane, int w) {
            const int fa = FM * (w / WCOLS), fb = FN * (w % WCOLS);
            a_at = lds_addr(lds) + TA::read_base(lane) + TA::read_imm(1, 0) * (uint32_t)fa;
            b_at = lds_addr(lds) + A_BYTES + (uint32_t)(fb / 8) * TB::BYTES + TB::read_base(lane) +
                   TB::read_imm(1, 0) * (uint32_t)(fb % 8);
        }
        // A phase's matrix instructions, from `stage`.
        __device__ __forceinline__ void multiply(int stage, floatx4 (&acc)[FM][FN]) const {
            const uint32_t sa = a_at + (uint32_t)(stage * STAGE), sb = b_at + (uint32_t)(stage * STAGE);
            u32x4 aq[FM], bq[FN];
            u32x2 ah[FM][2], bh[FN][2];
            if constexpr (KCA) {
#pragma unroll
                for (int i = 0; i < FM; ++i) aq[i] = lds_read128(sa + TA::read_imm(i, 0));
            } else {
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) ah[i][h] = read_tr16_off(sa, (int)TA::read_imm(i, h));
            }
            if constexpr (KCB) {
#pragma unroll
                for (int i = 0; i < FN; ++i) bq[i] = lds_read128(sb + TB::read_imm(i, 0));
            } else {
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) bh[i][h] = read_tr16_off(sb, (int)TB::read_imm(i, h));
            }
            if constexpr (!KCA) {
                wait_halves(ah);
#pragma unroll
                for (int i = 0; i < FM; ++i) aq[i] = u32x4{ah[i][0][0], ah[i][0][1], ah[i][1][0], ah[i][1][1]};
            }
            if constexpr (!KCB) {
                wait_halves(bh);
#pragma unroll
                for (int i = 0; i < FN; ++i) bq[i] = u32x4{bh[i][0][0], bh[i][0][1], bh[i][1][0], bh[i][1][1]};
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = KCA ? mfma16x16<FMT>(aq[i], bq[j], acc[i][j]) : mfma16x16<FMT>(bq[j], aq[i], acc[i][j]);
        }
    };
    __device__ static __forceinline__ void clear(floatx4 (&acc)[FM][FN]) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    }

    // The tile at (m0, n0) of the product; K > 0 if DIRECT.  turn: the phase to begin
    // with, modulo their number (the others follow, then those before it), only for
    // a direct product without k-contiguous factors.
    __device__ static __forceinline__ void run(const Gemm16Args& p, int m0, int n0, unsigned char* lds,
                                               floatx4 (&acc)[FM][FN], int turn = 0) {
        if constexpr (DIRECT) run_direct(p, m0, n0, lds, acc, turn);
        else run_staged(p, m0, n0, lds, acc);
    }

    // Zeros over the values from k on in the runs that hold the last phase's k (not
    // a multiple of 8) of k-contiguous factors: what was copied there lies past K.
    __device__ static __forceinline__ void cut_runs(unsigned char* stage, int k) {
        u32x4 mask;
#pragma unroll
        for (int d = 0; d < 4; ++d)
            mask[d] = (2 * d < k % 8 ? 0x0000FFFFu : 0u) | (2 * d + 1 < k % 8 ? 0xFFFF0000u : 0u);
        auto cut = [&](unsigned char* tile, int rows) __attribute__((always_inline)) {
            for (int r = threadIdx.x; r < rows; r += 256)
                *reinterpret_cast<u32x4*>(tile + 64 * r + 16 * ((k / 8) ^ (((r >> 3) & 1) << 1))) &= mask;
        };
        if constexpr (KCA) cut(stage, BM);
        if constexpr (KCB) cut(stage + A_BYTES, BN);
        __syncthreads();
    }

    __device__ static __forceinline__ void run_direct(const Gemm16Args& p, int m0, int n0, unsigned char* lds,
                                                      floatx4 (&acc)[FM][FN], int turn) {
        const int lane = threadIdx.x & 63;
        const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        // This wave's copies: CA of A's, CB of those of one 128-wide half of B's
        // columns.  Offsets are past the end by themselves wherever zeros are
        // wanted: rows past the last one, k past K of a k-contiguous factor (the
        // last phase), rows k past K of the other kind.
        constexpr uint32_t kPastEnd = 0x80000000u;
        const int half = CB * w / 8, b0 = CB * w % 8;
        uint32_t offset[COPIES];
#pragma unroll
        for (int j = 0; j < CA; ++j) offset[j] = (uint32_t)TA::copy_src(CA * w + j, lane, m0, p.lda);
#pragma unroll
        for (int j = 0; j < CB; ++j) offset[CA + j] = (uint32_t)TB::copy_src(b0 + j, lane, n0 + 128 * half, p.ldb);
        constexpr int kRawBufferWord3 = 0x00020000;
        const int64_t a_rows = KCA ? p.M : p.K, a_cols = KCA ? p.K : p.M;
        const int64_t b_rows = KCB ? p.N : p.K, b_cols = KCB ? p.K : p.N;
        const __amdgpu_buffer_rsrc_t rsrc_a = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(p.A), (short)0, (int)(2 * ((a_rows - 1) * p.lda + a_cols)), kRawBufferWord3);
        const __amdgpu_buffer_rsrc_t rsrc_b = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(p.B), (short)0, (int)(2 * ((b_rows - 1) * p.ldb + b_cols)), kRawBufferWord3);
        auto copies = [&](int ph, int stage) __attribute__((always_inline)) {
            const int k0 = BK * ph;
            const bool last = k0 + BK > p.K;
            unsigned char* const at = lds + stage * STAGE;
            const uint32_t pa = (uint32_t)TA::phase_bytes(k0, p.lda), pb = (uint32_t)TB::phase_bytes(k0, p.ldb);
#pragma unroll
            for (int j = 0; j < CA; ++j) {
                uint32_t v = offset[j] + pa;
                if (KCA && last && k0 + TA::copy_k(CA * w + j, lane) >= p.K) v = kPastEnd;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc_a, (__attribute__((address_space(3))) void*)(at + TA::copy_dst(CA * w + j)), 16, (int)v, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < CB; ++j) {
                uint32_t v = offset[CA + j] + pb;
                if (KCB && last && k0 + TB::copy_k(b0 + j, lane) >= p.K) v = kPastEnd;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc_b,
                    (__attribute__((address_space(3))) void*)(at + A_BYTES + half * TB::BYTES + TB::copy_dst(b0 + j)), 16,
                    (int)v, 0, 0, 0);
            }
        };
        const Fragments fragments(lds, lane, w);
        clear(acc);
        const int phases = ceil_div(p.K, BK);
        constexpr bool TURNS = !KCA && !KCB && NB == 2;
        if constexpr (TURNS) turn %= phases;
        auto turned = [&](int ph) __attribute__((always_inline)) {
            return !TURNS ? ph : ph + turn < phases ? ph + turn : ph + turn - phases;
        };
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s)
            if (s < phases) copies(turned(s), s);
        int stage = 0;
        for (int ph = 0; ph < phases; ++ph) {
            // This phase's copies of this wave have landed (those of the next ones
            // may be in flight) and its reads of the phase before are done; then
            // everyone's are, and the stage before is free.
            wait_phase<STAGES - 2, COPIES>(phases - 1 - ph);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (ph + STAGES - 1 < phases) copies(turned(ph + STAGES - 1), stage == 0 ? STAGES - 1 : stage - 1);
            if ((KCA || KCB) && ph == phases - 1 && p.K % 8 != 0) cut_runs(lds + stage * STAGE, p.K % 32);
            fragments.multiply(stage, acc);
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        }
        __syncthreads();                               // the stages are free
    }

    // Through registers, for operands anywhere in memory.  A run is one load of 16
    // bytes without a branch: rows past the last one repeat it and columns past
    // the last one repeat the first (both end in results that are not stored), and
    // a run across the last column reads on into the next row.  Only the last
    // phase, which holds the last row and K's edge, takes its values one by one
    // with zeros past K; it is computed first.  Rows shorter than a run (of an
    // operand whose k runs along its columns) always go one by one.
    __device__ static __forceinline__ void run_staged(const Gemm16Args& p, int m0, int n0, unsigned char* lds,
                                                      floatx4 (&acc)[FM][FN]) {
        const int lane = threadIdx.x & 63;
        const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const int half = CB * w / 8, b0 = CB * w % 8;
        const Fragments fragments(lds, lane, w);
        clear(acc);
        const int phases = ceil_div(p.K, BK);
        if (phases == 0) return __syncthreads();
        constexpr int AHEAD = 3;
        u32x4 held[AHEAD][COPIES];
        // Copy j's first value at phase 0, the first of its k and how many values
        // of a run of the other kind exist.
        const uint16_t* at[COPIES];
        int k_of[COPIES], width[COPIES];
        auto place = [&](int j, bool kc, const uint16_t* base, int64_t ld, int size, int mn, int k) __attribute__((always_inline)) {
            const int row = min(mn, size - 1), col = mn < size ? mn : 0;
            at[j] = base + (kc ? (int64_t)row * ld + k : (int64_t)k * ld + col);
            k_of[j] = k;
            width[j] = kc ? 8 : min(size - col, 8);
        };
#pragma unroll
        for (int j = 0; j < CA; ++j)
            place(j, KCA, p.A, p.lda, p.M, m0 + TA::copy_mn(CA * w + j, lane), TA::copy_k(CA * w + j, lane));
#pragma unroll
        for (int j = 0; j < CB; ++j)
            place(CA + j, KCB, p.B, p.ldb, p.N, n0 + 128 * half + TB::copy_mn(b0 + j, lane), TB::copy_k(b0 + j, lane));
        const int64_t step_a = BK * (KCA ? 1 : p.lda), step_b = BK * (KCB ? 1 : p.ldb);
        const bool short_a = !KCA && p.lda < 8, short_b = !KCB && p.ldb < 8;
        // The values of copy j's run in phase ph, one by one.
        auto single = [&](int j, int ph) __attribute__((always_inline)) -> u32x4 {
            const bool kc = j < CA ? KCA : KCB;
            const int left = p.K - BK * ph - k_of[j];                     // of k, from the run's first
            const int valid = kc ? min(left, 8) : left > 0 ? width[j] : 0;
            const uint16_t* const q = valid > 0 ? at[j] + ph * (j < CA ? step_a : step_b) : j < CA ? p.A : p.B;
            unsigned u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = q[max(min(e, valid - 1), 0)];
            u32x4 v;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                v[d] = (2 * d < valid ? u[2 * d] : 0u) | (2 * d + 1 < valid ? u[2 * d + 1] << 16 : 0u);
            return v;
        };
        auto load = [&](int ph, u32x4 (&v)[COPIES]) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < COPIES; ++j) {
                if (j < CA ? short_a : short_b) v[j] = single(j, ph);
                else __builtin_memcpy(&v[j], at[j] + ph * (j < CA ? step_a : step_b), 16);
            }
        };
        auto store = [&](const u32x4 (&v)[COPIES], int stage) __attribute__((always_inline)) {
            unsigned char* const to = lds + stage * STAGE + 16 * lane;
#pragma unroll
            for (int j = 0; j < CA; ++j) *reinterpret_cast<u32x4*>(to + TA::copy_dst(CA * w + j)) = v[j];
#pragma unroll
            for (int j = 0; j < CB; ++j)
                *reinterpret_cast<u32x4*>(to + A_BYTES + half * TB::BYTES + TB::copy_dst(b0 + j)) = v[CA + j];
        };
        // Position 0 is the last phase, position i phase i - 1.
#pragma unroll
        for (int s = 1; s < AHEAD; ++s)
            if (s < phases) load(s - 1, held[s]);
#pragma unroll
        for (int j = 0; j < COPIES; ++j) held[0][j] = single(j, phases - 1);
        for (int i = 0; i < phases; i += AHEAD) {
#pragma unroll
            for (int s = 0; s < AHEAD; ++s) {
                if (i + s >= phases) break;
                const int stage = (i + s) & 1;
                // The stage's readers, two phases ago, passed the last barrier.
                store(held[s], stage);
                if (i + s + AHEAD < phases) load(i + s + AHEAD - 1, held[s]);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                fragments.multiply(stage, acc);
            }
        }
        __syncthreads();
    }
    __device__ static __forceinline__ void wait_halves(u32x2 (&h)[8][2]) { wait_tied(h); }
    __device__ static __forceinline__ void wait_halves(u32x2 (&h)[4][2]) {
        asm volatile("s_waitcnt lgkmcnt(0)"
                     : "+v"(h[0][0]), "+v"(h[0][1]), "+v"(h[1][0]), "+v"(h[1][1]), "+v"(h[2][0]), "+v"(h[2][1]),
                       "+v"(h[3][0]), "+v"(h[3][1])
                     :
                     : "memory");
    }

    __device__ static __forceinline__ u32x4 pack(const float (&v)[8]) {
        using T = typename Stored<FMT>::T;
        T raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = (T)v[i];
        u32x4 d;
        __builtin_memcpy(&d, raw, 16);
        return d;
    }

    // The forward epilogue; thread t holds bias value n0 + t.  streamed: C's whole
    // runs go past the caches.
    __device__ static __forceinline__ void finish(const floatx4 (&acc)[FM][FN], const EpilogueArgs& e, int m0, int n0,
                                                  float bias, bool streamed, unsigned char* lds) {
        const int lane = threadIdx.x & 63;
        const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        float* const shared = reinterpret_cast<float*>(lds + BIAS);
        if ((int)threadIdx.x < BN) shared[threadIdx.x] = bias;
        __syncthreads();
        float* const patch = reinterpret_cast<float*>(lds) + w * Staged::PATCH;
        const int row0 = m0 + 16 * FM * (w / WCOLS), wcol = 16 * FN * (w % WCOLS), col0 = n0 + wcol;
        auto bias_of = [&](int col, float (&b)[8]) __attribute__((always_inline)) {
            const floatx4 lo = *reinterpret_cast<const floatx4*>(shared + wcol + col);
            const floatx4 hi = *reinterpret_cast<const floatx4*>(shared + wcol + col + 4);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                b[c] = lo[c];
                b[4 + c] = hi[c];
            }
        };
        // Whole runs at places of 32 bits from the wave's corner; else value by
        // value where a run crosses N, with what the epilogue reads.
        constexpr int64_t kMaxLd = 1 << 22;
        if ((n0 + BN <= e.N || e.N % 8 == 0) && e.residual == nullptr && e.ldc < kMaxLd &&
            (e.preact == nullptr || e.ldz < kMaxLd)) {
            char* const c_base = static_cast<char*>(e.C) + (e.c_type == 2 ? 4 : 2) * ((int64_t)row0 * e.ldc + col0);
            char* const z_base = static_cast<char*>(e.preact) + 2 * ((int64_t)row0 * e.ldz + col0);
            const unsigned ldc = (unsigned)e.ldc, ldz = (unsigned)e.ldz;
            Staged::template rows<false, 0>(
                acc, patch, nullptr, lane, false, [](int, int, u32x4 (&)[1]) {},
                [&](int row, int col, float (&v)[8], const u32x4 (&)[1]) __attribute__((always_inline)) {
                    if (row0 + row >= e.M || col0 + col >= e.N) return;
                    float b[8];
                    bias_of(col, b);
                    const Run run{};
                    const uint32_t c_at = __umul24(row, ldc) + col, z_at = __umul24(row, ldz) + col;
                    if (!streamed) return run.finish_at(e, c_base, c_at, z_base, z_at, b, v);
                    run.apply(
                        e, b, v,
                        [&](const float (&z)[8]) __attribute__((always_inline)) {
                            Run::template store_whole<FMT>(z_base, 2 * z_at, z);
                        },
                        [&](const float (&q)[8]) __attribute__((always_inline)) {
                            store_streamed(c_base + 2 * c_at, pack(q));
                        });
                },
                [](int, int) {});
        } else {
            Staged::template rows<false, 0>(
                acc, patch, nullptr, lane, false, [](int, int, u32x4 (&)[1]) {},
                [&](int row, int col, float (&v)[8], const u32x4 (&)[1]) __attribute__((always_inline)) {
                    if (row0 + row >= e.M || col0 + col >= e.N) return;
                    float b[8];
                    bias_of(col, b);
                    Run run;
                    run.load(e, row0 + row, col0 + col);
                    run.finish(e, row0 + row, col0 + col, b, v);
                },
                [](int, int) {});
        }
    }

    // The gradient's, which stores its sums.  Register r of acc[i][j] of lane (c =
    // l % 16, g = l / 16) is row 16 i + c, column 16 j + 4 g + r of the wave's
    // span (the matrix instruction gets B's fragment first): a lane's 4 values of
    // two blocks j, j + 1 become 8 consecutive ones of one by a swap of the lane
    // groups' halves, and a store of 16 bytes a lane writes 64 bytes of 16 rows.
    // planes: into binary32 planes of a sum still to be joined.  Whole lines of the
    // gradient go past the caches, which hold what the other blocks read: 8192 x
    // 2048 x 4096 over 16 groups 150 us against 204 with ordinary stores (4096 x
    // 1024 x 2048 over 64 68 against 117); through LDS, as runs of 256 bytes, 158
    // and 75.  That is with its factors in the last-level cache; within a backward
    // pass they come from memory, and it gains less: the pass over 2048 x 512 x
    // 1024 and 64 groups 47 us against 57, 1024 x 4096 x 4096 and 8 215 against 232,
    // 8192 x 2048 x 4096 and 16 391 against 400.  Parts of lines go through the
    // caches: 2000 x 1000 x 1000 over 4 15.3 us against 16.
    __device__ static __forceinline__ void finish_gradient(const floatx4 (&acc)[FM][FN], const EpilogueArgs& e, int m0,
                                                           int n0, bool planes, unsigned char* lds) {
        const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
        const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const int row0 = m0 + 16 * FM * (w / WCOLS), col0 = n0 + 16 * FN * (w % WCOLS);
        if (row0 >= e.M || col0 >= e.N) return;
        const int size = e.c_type == 2 ? 4 : 2;
        if (e.N % 8 != 0 || (size * e.ldc | (int64_t)(uintptr_t)e.C) % 16 != 0)
            return gradient_runs(acc, e, row0, col0, planes, lds);
        const bool streamed = !planes && (size * e.ldc | (int64_t)(uintptr_t)e.C) % 64 == 0;
        const int to = 16 * (g & 1) + 8 * (g >> 1);        // the 8 columns of a pair of blocks a lane stores
        auto put = [&](int row, int col, u32x4 v) __attribute__((always_inline)) {
            if (row >= e.M || col >= e.N) return;
            char* const p = static_cast<char*>(e.C) + size * (row * e.ldc + col);
            if (streamed) store_streamed(p, v);
            else __builtin_memcpy(p, &v, 16);
        };
#pragma unroll
        for (int j = 0; j < FN; j += 2) {
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int row = row0 + 16 * i + c, col = col0 + 16 * j;
                if (e.c_type == 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) put(row, col + 16 * h + 4 * g, __builtin_bit_cast(u32x4, acc[i][j + h]));
                    continue;
                }
                const floatx4 a = acc[i][j], b = acc[i][j + 1];
                const u32x4 d = pack({a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
                const auto lo = __builtin_amdgcn_permlane16_swap(d[0], d[2], false, false);
                const auto hi = __builtin_amdgcn_permlane16_swap(d[1], d[3], false, false);
                put(row, col + to, u32x4{lo[0], hi[0], lo[1], hi[1]});
            }
        }
    }

    // The same where rows do not begin at 16 bytes: 16 rows at a time through the
    // wave's patch of LDS, as runs of 8 columns, a wave's span of a row at once
    // (8192 x 2001 x 2003 over 16 groups 154 us against 188 from the registers).
    __device__ static __forceinline__ void gradient_runs(const floatx4 (&acc)[FM][FN], const EpilogueArgs& e, int row0,
                                                         int col0, bool planes, unsigned char* lds) {
        const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
        float* const patch = reinterpret_cast<float*>(lds) + (threadIdx.x >> 6) * Staged::PATCH;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int j = 0; j < FN; ++j) *reinterpret_cast<floatx4*>(patch + c * Staged::PITCH + 16 * j + 4 * g) = acc[i][j];
            wave_lds_fence();
#pragma unroll
            for (int t = 0; t < FN / 2; ++t) {
                const int k = 64 * t + lane, row = row0 + 16 * i + k / (2 * FN), at = 8 * (k % (2 * FN)), col = col0 + at;
                const floatx4* const q = reinterpret_cast<const floatx4*>(patch + k / (2 * FN) * Staged::PITCH + at);
                const floatx4 lo = q[0], hi = q[1];
                const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                if (row >= e.M || col >= e.N) continue;
                const int64_t index = row * e.ldc + col;
                if (e.c_type == FMT && !planes && col + 8 <= e.N) store_streamed(static_cast<char*>(e.C) + 2 * index, pack(v));
                else store_values(e.c_type, e.C, index, e.N - col, v);
            }
            wave_lds_fence();
        }
    }
};

// Blocks (x, y) of one x split K: y takes k from y k_share on (a multiple of 32)
// and stores its sums as plane y, `plane` floats after the one before (then e is
// that matrix, without a layer's epilogue); k_share = K: not split.
// The 128 x 256 tiles past whole rounds of the 512 that the chip holds would run
// alone on their CUs, at half its rate; a quarter of a round or less of them goes
// to four times the blocks of 64 x 128, whose six stages take no more LDS: 8192 x
// 2048 x 4096 over 16 groups with transposed weights 192 us against 221, 16384 x
// 4096 x 4096 over 8 544 against 560 (up to half a round: 12000 x 4096 x 4096 over
// 8 388 us against 404, but 5000 213 against 199 and 9000 323 against 311).  Not
// where K is split: there one round holds every block.
constexpr bool quarters(int bm, int nb, bool direct) { return direct && bm == 128 && nb == 2; }
constexpr int kRound = 512;

template <int FMT, bool KCB, int BM, int NB, int STAGES, int BLOCKS, bool DIRECT>
__global__ __launch_bounds__(256, BLOCKS)
void grouped_shared_kernel(GroupedArgs a, Gemm16Args p, EpilogueArgs e, int tiles_n, int group_m, int k_share,
                           int64_t plane, bool streamed) {
    using Core = GroupedSharedCore<FMT, true, KCB, BM, NB, STAGES, BLOCKS, DIRECT>;
    constexpr bool QUARTERS = quarters(BM, NB, DIRECT);
    using Quarter = GroupedSharedCore<FMT, true, KCB, 64, 1, QUARTERS ? 6 : 2, 2, DIRECT>;
    constexpr int LDS_BYTES = QUARTERS && Quarter::LDS_BYTES > Core::LDS_BYTES ? Quarter::LDS_BYTES : Core::LDS_BYTES;
    __shared__ __attribute__((aligned(16))) unsigned char lds[LDS_BYTES];
    const GroupRows r = locate_group_tile<BM>(a, (int)blockIdx.x, tiles_n, group_m, QUARTERS && gridDim.y == 1 ? kRound : 0);
    if (r.rows < 0) return;
    enter_group(a, r, &p, &e);
    int m0 = BM * r.tm, n0 = Core::BN * r.tn;
    if constexpr (QUARTERS) {
        if (r.quarter >= 0) {
            m0 += 64 * (r.quarter >> 1);
            n0 += 128 * (r.quarter & 1);
            if (m0 >= r.rows || n0 >= p.N) return;
            p.A += (int64_t)m0 * p.lda;
            p.M = min(r.rows - m0, 64);
            float bias[1] = {0.0f};
            if ((int)threadIdx.x < Quarter::BN) load_bias(e, n0 + (int)threadIdx.x, bias);
            floatx4 acc[Quarter::FM][Quarter::FN];
            Quarter::run(p, 0, n0, lds, acc);
            return Quarter::finish(acc, e, m0, n0, bias[0], streamed, lds);
        }
    }
    p.A += (int64_t)m0 * p.lda;
    p.M = min(r.rows - m0, BM);
    const int k0 = (int)blockIdx.y * k_share;
    p.A += k0;
    p.B += KCB ? (int64_t)k0 : k0 * p.ldb;
    p.K = min(p.K - k0, k_share);
    e.C = static_cast<char*>(e.C) + 4 * (blockIdx.y * plane);
    float bias[1] = {0.0f};
    if ((int)threadIdx.x < Core::BN) load_bias(e, n0 + (int)threadIdx.x, bias);
    floatx4 acc[Core::FM][Core::FN];
    Core::run(p, 0, n0, lds, acc);
    Core::finish(acc, e, m0, n0, bias[0], streamed, lds);
}

// The same for the gradient: the group's rows in gridDim.y shares.
// Where 128 x 256 tiles make more than four rounds, neighbouring tiles begin at
// different rows, so that blocks which start together do not ask for the same
// lines at once (8192 x 4096 x 4096 over 16 groups 337 us against 378, over 8 270
// against 285, 16384 x 4096 x 4096 over 16 542 against 583, over 8 480 against 487 to
// 495; 4096 x 4096 x 4096 over 8 149 against 148).  Fewer rounds lose what they share in
// the L2s (4096 x 4096 x 4096 in one 110 us against 104, over 4 128 against 124).  The
// sums' order then depends on the tile's place, the same in every call.
template <int FMT, int NB, int STAGES, int BLOCKS, bool DIRECT>
__global__ __launch_bounds__(256, BLOCKS)
void grouped_grad_shared_kernel(GroupedArgs a, Gemm16Args p, EpilogueArgs e, int tiles_m, int tiles_n, int group_m,
                                int64_t plane) {
    using Core = GroupedSharedCore<FMT, false, false, 128, NB, STAGES, BLOCKS, DIRECT>;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Core::LDS_BYTES];
    GroupRows r = locate_grad_tile(a, (int)blockIdx.x, tiles_m, tiles_n, group_m);
    const int splits = (int)gridDim.y;
    const RowShare share = row_share(r.rows, splits, (int)blockIdx.y);
    r.begin += share.first;
    r.rows = share.rows;
    enter_grad_group(a, r, &p, &e);
    e.C = static_cast<char*>(e.C) + 4 * (blockIdx.y * plane);
    const int m0 = Core::BM * r.tm, n0 = Core::BN * r.tn;
    if (r.rows == 0) return zero_tile<Core::BM, Core::BN>(e, m0, n0);
    floatx4 acc[Core::FM][Core::FN];
    Core::run(p, m0, n0, lds, acc, NB == 2 && gridDim.x > 4 * kRound ? r.tm + r.tn : 0);
    Core::finish_gradient(acc, e, m0, n0, splits > 1, lds);
}

// Outputs from here on go past the caches (a quarter of the 32 MB of the L2s: they
// would push the operands out).  4096 x 2044 x 2044 over 8 groups 65 us against 78
// with ordinary stores, 16384 x 4096 x 4096 over 8 558 against 567; 16 x 2048 x
// 4096 over 16 42 against 41.
constexpr int64_t kStreamedValues = 4 << 20;

template <int BM, int NB, int STAGES, int BLOCKS, bool DIRECT>
void launch(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format, int op_b,
            int k_share, int64_t plane) {
    constexpr int kGroupM = 1024 / BM;
    const bool streamed = DIRECT && e.c_type == format && (int64_t)a.rows * p.N >= kStreamedValues;
    const int tn = ceil_div(p.N, 128 * NB);
    const int64_t tiles = grouped_row_tiles(a.rows, a.groups, BM) * tn;
    const int shares = p.K > 0 ? ceil_div(p.K, k_share) : 1;
    const int64_t more = quarters(BM, NB, DIRECT) && shares == 1 ? 3 * std::min<int64_t>(tiles, kRound / 4) : 0;
    const dim3 g((unsigned)(tiles + more), (unsigned)shares), b(256);
    auto run = [&](auto fmt, auto kcb) {
        hipLaunchKernelGGL((grouped_shared_kernel<decltype(fmt)::value, decltype(kcb)::value, BM, NB, STAGES, BLOCKS,
                                                  DIRECT>), g, b, 0, s, a, p, e, tn, kGroupM, k_share, plane, streamed);
    };
    if (format == 0 && op_b) run(std::integral_constant<int, 0>{}, std::true_type{});
    else if (format == 0) run(std::integral_constant<int, 0>{}, std::false_type{});
    else if (op_b) run(std::integral_constant<int, 1>{}, std::true_type{});
    else run(std::integral_constant<int, 1>{}, std::false_type{});
}

template <int NB, int STAGES, int BLOCKS, bool DIRECT>
void launch_grad(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format,
                 int splits, int64_t plane) {
    constexpr int kGroupM = 8;
    const int tm = ceil_div(p.M, 128), tn = ceil_div(p.N, 128 * NB);
    const dim3 g((unsigned)(tm * tn * a.groups), (unsigned)splits), b(256);
    if (format == 0)
        hipLaunchKernelGGL((grouped_grad_shared_kernel<0, NB, STAGES, BLOCKS, DIRECT>), g, b, 0, s, a, p, e, tm, tn, kGroupM, plane);
    else
        hipLaunchKernelGGL((grouped_grad_shared_kernel<1, NB, STAGES, BLOCKS, DIRECT>), g, b, 0, s, a, p, e, tm, tn, kGroupM, plane);
}

}  // namespace

hipError_t launch_grouped_shared(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                                 int format, int op_b, bool direct, int bm, int bn, int k_share, int64_t plane) {
    if (!direct) {
        if (bm == 128) launch<128, 1, 2, 2, false>(a, p, e, s, format, op_b, k_share, plane);
        else launch<64, 1, 2, 3, false>(a, p, e, s, format, op_b, k_share, plane);
    } else if (bm == 128 && bn == 256) launch<128, 2, 3, 2, true>(a, p, e, s, format, op_b, k_share, plane);
    else if (bm == 128) launch<128, 1, 3, 3, true>(a, p, e, s, format, op_b, k_share, plane);
    else if (bn == 256) launch<64, 2, 3, 2, true>(a, p, e, s, format, op_b, k_share, plane);
    else launch<64, 1, 4, 3, true>(a, p, e, s, format, op_b, k_share, plane);
    return hipGetLastError();
}

hipError_t launch_grouped_grad_shared(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                                      int format, bool direct, int bn, int splits, int64_t plane) {
    if (!direct) launch_grad<1, 2, 2, false>(a, p, e, s, format, splits, plane);
    else if (bn == 256) launch_grad<2, 3, 2, true>(a, p, e, s, format, splits, plane);
    else launch_grad<1, 3, 3, true>(a, p, e, s, format, splits, plane);
    return hipGetLastError();
}

}  // namespace gemmf32
