// mfma16_ksplit.hip -- the mixed-precision product (bfloat16 or binary16
// factors, binary32 accumulation) for few output tiles and long K.
//
// The one-volume PMPP notes run the fully connected layer as a matrix
// product on matrix units fed FP16 or BF16 and accumulating in FP32
// (deep-learning chapter, "FC Layer = GEMM", "Mixed Precision"); this is
// that product with the tiled structure of the pages' shared-memory chapter
// (tiles staged in LDS, ghost zeros past the matrix edges, a guarded store),
// for the shapes whose large tiles would leave most compute units idle.
//
// Built with the matrix instructions' vector-register form
// (-mllvm -amdgpu-mfma-vgpr-form=true, see build.py): with the accumulators
// in AGPRs the register allocator copied every accumulator before each
// matrix instruction of this kernel.
#include "mfma16_ksplit_core.h"

namespace gemmf32 {

namespace {

// Few output tiles, long K: 64 x 64 tiles, one per block, whose four waves
// each compute the whole tile over every fourth 32-deep phase (wave w:
// phases w, w + 4, ...) from LDS stages of their own, which only that wave
// copies into and reads; the four partial tiles meet in LDS at the end and
// are added in wave order (deterministic; the same bits for every op pair).
// A 1024 x 1024 x 4096 product has 16 tiles of 256 x 256 for 256 CUs; here
// it has 256 blocks.
//
// Matrix instruction v_mfma_f32_16x16x32_{bf16,f16}: lane l supplies
// A[l % 16][8 (l / 16) .. + 7] and B[8 (l / 16) .. + 7][l % 16]; accumulator
// register r holds D[4 (l / 16) + r][l % 16].  A wave's 64 x 64 tile is 4 x 4
// blocks of 16 x 16; a 32-deep phase is one step of 16 instructions, about
// 256 clocks of the matrix core, so each wave keeps four stages (8 KB each,
// 128 KB per block) and copies a phase three phases ahead of its use.  The
// phase loop is unrolled by the four stages, so every stage offset is an
// instruction offset: besides the matrix instructions the loop holds only
// the fragment reads and the copies (buffer loads into LDS whose phase is in
// the scalar offset).
//
// Tiles (per stage):
//   KC (k-contiguous factor: A as stored, B stored transposed): 64 rows of
//      32 k (64 bytes), the 16-byte chunk c (8 k) of row r at
//      c ^ (2 ((r / 8) mod 2)); a 1 KB copy fills 16 rows; a fragment is one
//      128-bit read of row 16 f + l % 16, chunk l / 16.  A 128-bit read
//      serves, per half-wave, the 4-lane quads of even index parity in one
//      cycle (lanes 0-3, 12-15, 20-23, 24-27) and the others in the next
//      (measured on MI355X); those 16 lanes hit 16 different 4-bank groups.
//   MC (mn-contiguous factor: B as stored, A stored transposed): 32 k rows
//      of 64 values (128 bytes), chunk c of row r at
//      c ^ (2 ((r / 2) mod 2) + 4 ((r / 8) mod 2)); a copy fills 8 rows; a
//      fragment is two ds_read_b64_tr_b16 reads (k 0..3 and 4..7 of the lane
//      group's eight), the 32 lanes of one read cycle over 8 rows and 16
//      different 4-bank groups.
//
// Phases are aligned to the end of K (K a multiple of 8), phase g covering
// k = K - 32 (P - g) .. + 31: only phase 0 can reach below k = 0, and its
// lanes there are pointed past the end of their buffer descriptor (zeros).
// Every copy that must bring zeros has a per-lane offset past the
// descriptor's end by itself (the scalar offset, which holds the phase,
// never decides it): rows of a KC factor past the tile's edge, and the
// 16-byte chunks of an MC factor wholly past its last column (in every
// phase).  A chunk of an MC factor across its last column reads the next
// row (only C entries outside the matrix use it), or, in the factor's last
// row -- in the last phase, whose per-lane offsets hold the phase (dlast) --
// its dwords up to the descriptor's end and zeros past it (the range check
// is per dword; the width is even, so no dword straddles the end).
template <int FMT, bool KCA, bool KCB>
__global__ __launch_bounds__(256)
void gemm16_ksplit_kernel(Gemm16Args p, int tiles_m, int tiles_n, int group_m) {
    using Core = KsplitCore<FMT, KCA, KCB>;
    __shared__ __attribute__((aligned(16))) uint16_t lds[Core::LDS_ELEMS];

    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int tm, tn;
    grouped_tile((int)blockIdx.x, tiles_m, tiles_n, group_m, &tm, &tn);
    const int m0 = tm * 64, n0 = tn * 64;
    Core::run(p, m0, n0, lds);

    // Wave v adds, in wave order, block row v: register r of block (v, j) of
    // lane l is row 16 v + 4 (l / 16) + r, column 16 j + l % 16 of the tile.
    const float* const part = reinterpret_cast<const float*>(lds);
    const int col_l = lane & 15, row_l = 4 * (lane >> 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = n0 + 16 * j + col_l;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float* q = part + ((4 * w + j) * 4 + r) * 64 + lane;
            const float v = ((q[0] + q[4096]) + q[2 * 4096]) + q[3 * 4096];
            const int row = m0 + 16 * w + row_l + r;
            if (row < p.M && col < p.N) p.C[(int64_t)row * p.ldc + col] = v;
        }
    }
}

}  // namespace

// The k-split kernel takes K a multiple of 8, an mn-contiguous factor's
// width even, vector-aligned operands (4-byte aligned bases, even leading
// dimensions) and operands below 2^31 bytes with a tile's overhang (32-bit
// offsets).
bool ksplit16_fits(const Gemm16Args& p, int op_a, int op_b) {
    const bool vec = ((reinterpret_cast<uintptr_t>(p.A) | reinterpret_cast<uintptr_t>(p.B)) & 3) == 0 &&
                     (p.lda % 2) == 0 && (p.ldb % 2) == 0;
    const int64_t a_rows = op_a ? p.K : p.M, b_rows = op_b ? p.N : p.K;
    const bool widths = (op_a == 0 || p.M % 2 == 0) && (op_b != 0 || p.N % 2 == 0);
    return vec && widths && p.K % 8 == 0 && p.K > 0 && p.M > 0 && p.N > 0 &&
           2 * (a_rows + 64) * p.lda < (1ll << 31) && 2 * (b_rows + 64) * p.ldb < (1ll << 31);
}
namespace {
template <int FMT, bool KCA, bool KCB>
hipError_t launch_ksplit16_kernel(const Gemm16Args& p, hipStream_t s, int tiles_m, int tiles_n, int group_m,
                                  unsigned blocks) {
    hipLaunchKernelGGL((gemm16_ksplit_kernel<FMT, KCA, KCB>), dim3(blocks), dim3(256), 0, s, p, tiles_m, tiles_n,
                       group_m);
    return hipGetLastError();
}
}  // namespace

// format: 0 bfloat16, 1 binary16; op_a / op_b: 1 if that factor is stored
// transposed.  64 x 64 tiles, tile-row groups of 8.
hipError_t launch_ksplit16(const Gemm16Args& p, hipStream_t s, int format, int op_a, int op_b) {
    const int tiles_m = ceil_div(p.M, 64), tiles_n = ceil_div(p.N, 64);
    const int64_t blocks = (int64_t)tiles_m * tiles_n;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
    const unsigned nb = (unsigned)blocks;
    switch (4 * (format ? 1 : 0) + 2 * (op_a ? 1 : 0) + (op_b ? 1 : 0)) {
        case 0: return launch_ksplit16_kernel<0, true, false>(p, s, tiles_m, tiles_n, 8, nb);
        case 1: return launch_ksplit16_kernel<0, true, true>(p, s, tiles_m, tiles_n, 8, nb);
        case 2: return launch_ksplit16_kernel<0, false, false>(p, s, tiles_m, tiles_n, 8, nb);
        case 3: return launch_ksplit16_kernel<0, false, true>(p, s, tiles_m, tiles_n, 8, nb);
        case 4: return launch_ksplit16_kernel<1, true, false>(p, s, tiles_m, tiles_n, 8, nb);
        case 5: return launch_ksplit16_kernel<1, true, true>(p, s, tiles_m, tiles_n, 8, nb);
        case 6: return launch_ksplit16_kernel<1, false, false>(p, s, tiles_m, tiles_n, 8, nb);
        default: return launch_ksplit16_kernel<1, false, true>(p, s, tiles_m, tiles_n, 8, nb);
    }
}


}  // namespace gemmf32
