// mfma16_wide.hip -- the scheduled 256 x 256 mixed-precision kernel
// (bfloat16 or binary16 factors, binary32 accumulation) on the 16 x 16 x 32
// matrix instruction.
//
// The one-volume PMPP notes run the fully connected layer as a matrix
// product on matrix units fed FP16 or BF16 and accumulating in FP32
// (deep-learning chapter, "FC Layer = GEMM", "Mixed Precision"); this is
// that product with the tiled structure of the pages' shared-memory chapter
// (tiles staged in LDS, ghost zeros past the matrix edges, a guarded store).
//
// Same block structure as gemm16_sched_kernel (mfma16.hip): 256 x 256 tiles,
// four waves (one per SIMD) of 128 x 128 each, 64-deep phases in two LDS
// stages, one barrier per phase, every instruction of the K loop placed in
// program order.  The instruction is v_mfma_f32_16x16x32 instead of
// 32 x 32 x 16: a wave's tile is 8 x 8 blocks of 16 x 16 and a phase is two
// 32-deep steps of 64 instructions (the same matrix-core clocks).  In a bare
// loop this form sustains a higher clock on MI355X than 32 x 32 x 16.
//
// The same kernel runs 192 x 192 tiles (template parameter BT): waves of 96
// x 96 (6 x 6 blocks), steps of 36 instructions, 6 copies per wave and phase
// for a k-contiguous factor (rows 0..191 of the layout below) and 8 for an
// mn-contiguous one (the layout below with each 512-byte k-row slot holding
// 192 values, the lanes of values 192..255 copying zeros).  Its copies need
// 42.7 bytes per clock per CU at the full matrix rate against 32 for 256 x
// 256 tiles: it is chosen only where its tile count fills the rounds of 256
// CUs much better.  Likewise 160 x 160 tiles: waves of 80 x 80 (5 x 5
// blocks), steps of 25 instructions, 5 copies per wave and phase for a
// k-contiguous factor and 8 for an mn-contiguous one (lanes of values
// 160..255 copying zeros); 51.2 bytes per clock per CU at the full matrix
// rate.
//
// The LDS tiles are laid out so that at most two per-lane bases per factor
// serve every fragment, step and read of a phase (all the rest are
// instruction offsets), and both kinds read without bank conflicts (64 banks
// of 4 bytes; measured):
//   KC (k-contiguous factor: A as stored, B stored transposed): 256 rows of
//      64 k (128 bytes), 16-byte chunk c (8 k) of row r at c ^ ((r / 2) mod
//      8), as in gemm16_sched_kernel.  A fragment (16 rows, 32 k) is one
//      128-bit read of row 16 f + l % 16, chunk 4 s + l / 16; the swizzle
//      depends on l % 16 only, so each step has one base and fragment f is
//      an instruction offset.  A 1 KB copy fills 8 rows.  (Rows of 32 k, 64
//      bytes, read this way conflict 2-way on gfx950 under every lane-to-
//      cycle grouping of 128-bit reads that agrees with the measured
//      conflict counts: the hardware does not serve lanes 0-15, 16-31, ...
//      together.)
//   MC (mn-contiguous factor: B as stored, A stored transposed): the stage is
//      32 pairs of 512-byte k rows, pair m at byte 1056 m (32 bytes of padding
//      after each pair); k row kappa of the phase (kappa = 32 s + 8 g + 4 h +
//      e: step s, lane group g, read h, e = 0..3) is row h of pair
//      e + 4 g + 16 s and holds the tile's 256 values in order.  A fragment
//      is two ds_read_b64_tr_b16 reads (h = 0, 1); the 8 rows one cycle reads
//      lie in pairs whose m mod 8 differ, each pair shifted by 8 banks
//      against the last.  A 1 KB copy fills one pair.
// Stage sizes: KC 32768 bytes, MC 33792; LDS holds A's two stages, then B's
// (at most 135168 bytes).
//
// Edge handling is that of gemm16_sched_kernel: each descriptor ends at its
// stored matrix's last element; a copy that must bring zeros has a per-lane
// offset past that end by itself (rows of a KC factor past the tile's edge
// in every phase; chunks or rows at k >= K in the last phase, whose copies
// take per-lane offsets with the phase folded in and a scalar offset of 0);
// the column overhang of an MC factor reads the next row (only C entries
// outside the matrix use it) or, in the last row, its dwords up to the end
// and zeros past it.  K need only be even: the one chunk per row of a KC
// factor that straddles K is copied whole, and its values past K are zeroed
// in the last phase's fragments.
//
// The k order inside each instruction (k = 32 s + 8 (l / 16) + e of lane l)
// does not depend on how a factor is stored, so the four op pairs give the
// same bits on explicitly transposed copies.
#include "mfma16_wide_core.h"

namespace gemmf32 {

namespace {

// BT: the tile's extent in M and N (256, or 192 or 160 for problems whose
// 256 x 256 tiles fill the CUs' rounds badly); each wave holds a quarter of
// it.
template <int FMT, bool KCA, bool KCB, int BT = 256>
__global__ __launch_bounds__(256)
void gemm16_wide_kernel(Gemm16Args p, int tiles_m, int tiles_n, int group_m) {
    using Core = WideCore<FMT, KCA, KCB, BT>;
    constexpr int FM = Core::FM, FN = Core::FN, WM = Core::WM, WN = Core::WN;
    __shared__ __attribute__((aligned(16))) unsigned char lds[Core::LDS_BYTES];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave / 2, wn = wave % 2;
    int tm, tn;
    grouped_tile((int)blockIdx.x, tiles_m, tiles_n, group_m, &tm, &tn);
    const int m0 = tm * BT, n0 = tn * BT;
    floatx4 acc[FM][FN];
    Core::run(p, m0, n0, lds, acc);

    // Guarded store (edge tiles run whole and store only what lies inside
    // C): register r of block (i, j) of lane l is row 16 i + 4 (l / 16) + r,
    // column 16 j + l % 16 of the wave's span.  Consecutive stores cover one
    // row across the blocks (512 contiguous bytes per lane group for a 256
    // tile; measured 1 % faster at 8192^3 than block by block).
    const int row0 = m0 + wm * WM + 4 * (lane >> 4), col0 = n0 + wn * WN + (lane & 15);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = row0 + 16 * i + r;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int col = col0 + 16 * j;
                if (row < p.M && col < p.N) p.C[(int64_t)row * p.ldc + col] = acc[i][j][r];
            }
        }
}

template <int FMT, bool KCA, bool KCB, int BT>
hipError_t launch_wide_kernel(const Gemm16Args& p, hipStream_t s, int tiles_m, int tiles_n, int group_m,
                              unsigned blocks) {
    hipLaunchKernelGGL((gemm16_wide_kernel<FMT, KCA, KCB, BT>), dim3(blocks), dim3(256), 0, s, p, tiles_m, tiles_n,
                       group_m);
    return hipGetLastError();
}

template <int BT>
hipError_t launch_wide_tiles(const Gemm16Args& p, hipStream_t s, int format, int op_a, int op_b, int group_m) {
    const int tiles_m = ceil_div(p.M, BT), tiles_n = ceil_div(p.N, BT);
    const int64_t blocks = (int64_t)tiles_m * tiles_n;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
    const unsigned nb = (unsigned)blocks;
    switch (4 * (format ? 1 : 0) + 2 * (op_a ? 1 : 0) + (op_b ? 1 : 0)) {
        case 0: return launch_wide_kernel<0, true, false, BT>(p, s, tiles_m, tiles_n, group_m, nb);
        case 1: return launch_wide_kernel<0, true, true, BT>(p, s, tiles_m, tiles_n, group_m, nb);
        case 2: return launch_wide_kernel<0, false, false, BT>(p, s, tiles_m, tiles_n, group_m, nb);
        case 3: return launch_wide_kernel<0, false, true, BT>(p, s, tiles_m, tiles_n, group_m, nb);
        case 4: return launch_wide_kernel<1, true, false, BT>(p, s, tiles_m, tiles_n, group_m, nb);
        case 5: return launch_wide_kernel<1, true, true, BT>(p, s, tiles_m, tiles_n, group_m, nb);
        case 6: return launch_wide_kernel<1, false, false, BT>(p, s, tiles_m, tiles_n, group_m, nb);
        default: return launch_wide_kernel<1, false, true, BT>(p, s, tiles_m, tiles_n, group_m, nb);
    }
}

}  // namespace

// K even and > 0 (the last phase's values past K are masked), an
// mn-contiguous factor's width (M for A stored transposed, N for B as
// stored) even, 4-byte aligned bases, even leading dimensions, and stored
// factors below 2^31 bytes with a tile's overhang.  Every descriptor then
// ends on a dword boundary: the range check is per dword, so with K odd the
// last row's last value would share a dword with the bytes past the end and
// read as zero.
bool wide_fits(const Gemm16Args& p, int op_a, int op_b) {
    const bool vec = ((reinterpret_cast<uintptr_t>(p.A) | reinterpret_cast<uintptr_t>(p.B)) & 3) == 0 &&
                     (p.lda % 2) == 0 && (p.ldb % 2) == 0;
    const int64_t a_rows = op_a ? p.K : p.M, b_rows = op_b ? p.N : p.K;
    const bool widths = (op_a == 0 || p.M % 2 == 0) && (op_b != 0 || p.N % 2 == 0);
    return vec && widths && p.K > 0 && p.K % 2 == 0 && p.M > 0 && p.N > 0 &&
           2 * (a_rows + 256) * p.lda < (1ll << 31) &&
           2 * (b_rows + 256) * p.ldb < (1ll << 31);
}

hipError_t launch_wide16(const Gemm16Args& p, hipStream_t s, int format, int op_a, int op_b, int group_m) {
    return launch_wide_tiles<256>(p, s, format, op_a, op_b, group_m);
}

hipError_t launch_wide16_192(const Gemm16Args& p, hipStream_t s, int format, int op_a, int op_b, int group_m) {
    return launch_wide_tiles<192>(p, s, format, op_a, op_b, group_m);
}

hipError_t launch_wide16_160(const Gemm16Args& p, hipStream_t s, int format, int op_a, int op_b, int group_m) {
    return launch_wide_tiles<160>(p, s, format, op_a, op_b, group_m);
}

}  // namespace gemmf32
