// mfma16_ksplit128.hip -- the mixed-precision product (bfloat16 or binary16
// factors, binary32 accumulation) for a few hundred output tiles of
// 128 x 128: one tile per block, its K split over the block's four waves.
//
// The one-volume PMPP notes run the fully connected layer as a matrix
// product on matrix units fed FP16 or BF16 and accumulating in FP32
// (deep-learning chapter, "FC Layer = GEMM", "Mixed Precision"); this is
// that product with the tiled structure of the pages' shared-memory chapter
// (tiles staged in LDS, ghost zeros past the matrix edges, a guarded store).
//
// A 2048^3 product has 64 tiles of 256 x 256 for 256 CUs, and 256 of
// 128 x 128: one round of one tile per CU.  Each of the block's four waves
// (one per SIMD) computes the whole 128 x 128 tile -- 8 x 8 blocks of
// 16 x 16 on v_mfma_f32_16x16x32, 256 accumulators -- over every fourth
// 32-deep phase (wave w: phases w, w + 4, ...) from two LDS stages of its
// own (16 KB each), which only that wave copies into and reads: no wave
// waits for another before the end, where the four partial tiles are added
// in wave order through LDS (deterministic; the same bits for every op
// pair).  A 128 x 128 tile needs 64 bytes of operands per clock at the
// matrix cores' full rate, about twice what a CU's L2 path brings, so the
// copies, not the instructions, set the pace.
//
// A phase is 64 matrix instructions (block (q / 8, q % 8) for instruction
// q, 1024 matrix-core clocks).  A wave runs its phases at positions: the
// last phase first, then (with an odd count) a position that copies zeros,
// then phases 0, 1, ..; at least two positions, an even number.  During
// position s it copies position s + 2 into the stage position s came from
// (16 copies of 1 KB, one after every odd instruction below 32), then, once
// the copies of position s + 1 have landed, reads position s + 1's fragments
// into its other register set (one read after each instruction from 24
// on).  The two phases that need per-lane copy offsets -- the last and the
// first -- sit at positions 0 to 2, copied in the prologue and by the first
// two positions (peeled); every later position runs one and the same body
// with one kind of copy, so the loop has no branch inside (a branch between
// phases keeps an unread register set live across it, and 256 accumulators
// leave no room for that).  Copies and reads aimed past the last position
// fill, and read, stages that nothing uses afterwards.

// Tiles (per stage, 128 mn x 32 k):
//   KC (k-contiguous factor: A as stored, B stored transposed): 128 rows of
//      32 k (64 bytes), the 16-byte chunk c (8 k) of row r at
//      c ^ (2 ((r / 8) mod 2)) (the 64 x 64 k-split kernel's rows); a 1 KB
//      copy fills 16 rows; fragment f is one 128-bit read of row
//      16 f + l % 16, chunk l / 16.
//   MC (mn-contiguous factor: B as stored, A stored transposed): 32 k rows
//      of 128 values (256 bytes) in eight groups of four, group Q at byte
//      1056 Q (32 bytes of padding a group); k row r = 8 g + 4 h + q (g =
//      0..3, h = 0..1, q = 0..3) is row 2 (g / 2) + h of group q + 4 (g mod
//      2).  A 1 KB copy fills one group; fragment f is two ds_read_b64_tr_b16
//      reads (h = 0, 1) of k rows 8 (l / 16) + 4 h + (l % 16) / 4.  The 32
//      lanes of one read cycle address 8 k rows in 8 different groups, each
//      shifted by 8 banks against the last (1056 = 33 x 32 bytes).
// Either way one read base per lane and factor serves every block, read and
// stage (instruction offsets).
//
// Edges as in the 64 x 64 k-split kernel: phases aligned to the end of K (K
// a multiple of 8), so only phase 0 reaches below k = 0; every copy that
// must bring zeros is past its descriptor's end by its per-lane offset
// alone (rows of a KC factor past the tile's edge, chunks of an MC factor
// wholly past its last column, lanes of phase 0 below k = 0, positions
// holding no phase); the wave's first and last phases take the phase in
// their per-lane offsets with a scalar offset of 0, so that a chunk of an
// MC factor's last row across its last column meets the descriptor's end by
// its own offset (the range check is per dword, and the width is even).
#include "mfma16_ksplit128_core.h"

namespace gemmf32 {

namespace {

template <int FMT, bool KCA, bool KCB>
__global__ __launch_bounds__(256)
void gemm16_ksplit128_kernel(Gemm16Args p, int tiles_m, int tiles_n, int group_m) {
    using Core = Ksplit128Core<FMT, KCA, KCB>;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Core::LDS_BYTES];
    int tm, tn;
    grouped_tile((int)blockIdx.x, tiles_m, tiles_n, group_m, &tm, &tn);
    const int m0 = tm * 128, n0 = tn * 128;
    floatx4 acc[8][8];
    Core::run(p, m0, n0, lds, acc);
    // One 128-bit store of the four values (32 lanes: 512 contiguous bytes of
    // a row of C).
    Core::exchange(
        acc, lds,
        [&](int, int, int r, int c4, floatx4 sum, float*) __attribute__((always_inline)) {
            const int row = m0 + r, col = n0 + c4;
            if (row >= p.M) return;
            float* const c = p.C + (int64_t)row * p.ldc + col;
            if (col + 3 < p.N && ((reinterpret_cast<uintptr_t>(c) & 15) == 0)) {
                *reinterpret_cast<floatx4*>(c) = sum;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < p.N) c[e] = sum[e];
            }
        },
        [](int) {});
}

template <int FMT, bool KCA, bool KCB>
hipError_t launch_ksplit128_kernel(const Gemm16Args& p, hipStream_t s, int tiles_m, int tiles_n, int group_m,
                                   unsigned blocks) {
    hipLaunchKernelGGL((gemm16_ksplit128_kernel<FMT, KCA, KCB>), dim3(blocks), dim3(256), 0, s, p, tiles_m, tiles_n,
                       group_m);
    return hipGetLastError();
}

}  // namespace

// K a multiple of 8, an mn-contiguous factor's width even, 4-byte aligned
// bases, even leading dimensions, and stored factors below 2^31 bytes with
// a tile's overhang (32-bit offsets).
bool ksplit128_fits(const Gemm16Args& p, int op_a, int op_b) {
    const bool vec = ((reinterpret_cast<uintptr_t>(p.A) | reinterpret_cast<uintptr_t>(p.B)) & 3) == 0 &&
                     (p.lda % 2) == 0 && (p.ldb % 2) == 0;
    const int64_t a_rows = op_a ? p.K : p.M, b_rows = op_b ? p.N : p.K;
    const bool widths = (op_a == 0 || p.M % 2 == 0) && (op_b != 0 || p.N % 2 == 0);
    return vec && widths && p.K % 8 == 0 && p.K > 0 && p.M > 0 && p.N > 0 &&
           2 * (a_rows + 128) * p.lda < (1ll << 31) && 2 * (b_rows + 128) * p.ldb < (1ll << 31);
}

// format: 0 bfloat16, 1 binary16; op_a / op_b: 1 if that factor is stored
// transposed.  128 x 128 tiles, tile-row groups of group_m.
hipError_t launch_ksplit128(const Gemm16Args& p, hipStream_t s, int format, int op_a, int op_b, int group_m) {
    const int tiles_m = ceil_div(p.M, 128), tiles_n = ceil_div(p.N, 128);
    const int64_t blocks = (int64_t)tiles_m * tiles_n;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
    const unsigned nb = (unsigned)blocks;
    switch (4 * (format ? 1 : 0) + 2 * (op_a ? 1 : 0) + (op_b ? 1 : 0)) {
        case 0: return launch_ksplit128_kernel<0, true, false>(p, s, tiles_m, tiles_n, group_m, nb);
        case 1: return launch_ksplit128_kernel<0, true, true>(p, s, tiles_m, tiles_n, group_m, nb);
        case 2: return launch_ksplit128_kernel<0, false, false>(p, s, tiles_m, tiles_n, group_m, nb);
        case 3: return launch_ksplit128_kernel<0, false, true>(p, s, tiles_m, tiles_n, group_m, nb);
        case 4: return launch_ksplit128_kernel<1, true, false>(p, s, tiles_m, tiles_n, group_m, nb);
        case 5: return launch_ksplit128_kernel<1, true, true>(p, s, tiles_m, tiles_n, group_m, nb);
        case 6: return launch_ksplit128_kernel<1, false, false>(p, s, tiles_m, tiles_n, group_m, nb);
        default: return launch_ksplit128_kernel<1, false, true>(p, s, tiles_m, tiles_n, group_m, nb);
    }
}

}  // namespace gemmf32
