// grouped_kernels.h -- the layer whose rows belong to groups (experts) with a
// weight each: where a block's tile lies, and the launchers of its kernels (not
// part of the public interface).
//
// Group g holds the rows offsets[g] .. offsets[g + 1] - 1 of A, sorted by
// group; the offsets are on the device, so the host knows only how many row
// tiles there can be and every block finds its own.  Offsets are read through
// clamps: whatever they hold, no row outside the matrices is touched.
#pragma once

#include "mfma16_common.h"

namespace gemmf32 {

// Rows x N = A (rows x K) W_g + bias_g, or, for the weights' gradient, M x N =
// A_g^T B_g.
struct GroupedArgs {
    int groups;
    const int* offsets;                // groups + 1
    int rows;                          // of A (and of B in the gradient)
    int64_t stride_b;                  // elements from a group's weight to the next; gradient: of C
    int64_t ld_bias;                   // elements from a group's bias to the next
};

// The smallest tile any launch uses: what the entry points bound the grid by.
constexpr int kGroupedSmallTile = 64;

// Row tiles of `tile` rows there can be: every group but the empty ones may
// leave one tile partly filled.
inline int64_t grouped_row_tiles(int64_t rows, int64_t groups, int64_t tile) {
    const int64_t used = groups < rows ? groups : rows;
    return (rows + used * (tile - 1)) / tile;
}

#if defined(__HIPCC__)
namespace {

// Share i of a group's rows among `splits` blocks: whole steps of 32 rows, the
// last ones cut off or empty.  Unsigned: rows reach 2^31 - 1, and no number here
// passes rows + 32 splits (a division in 64 bits costs 2 to 3 % of a small gradient).
struct RowShare {
    int first, rows;
};
__host__ __device__ __forceinline__ RowShare row_share(int rows, int splits, int i) {
    const unsigned all = rows, step = 32u * splits, share = (all + step - 1) / step * 32;
    const unsigned skip = i * share, first = skip < all ? skip : all;
    return {(int)first, (int)(share < all - first ? share : all - first)};
}

struct GroupRows {
    int group, begin, rows;            // of the group; rows < 0: none for this block
    int tm, tn;                        // the tile within the group
    int quarter;                       // of the tile; -1: all of it
};

__host__ __device__ __forceinline__ void group_range(const GroupedArgs& a, int g, int* begin, int* end) {
    const int from = a.offsets[g], to = a.offsets[g + 1];
    *begin = from < 0 ? 0 : from < a.rows ? from : a.rows;
    *end = to < *begin ? *begin : to < a.rows ? to : a.rows;
}

// Inclusive sum over the wave's lanes: within rows of 16 lanes, then across.
__device__ __forceinline__ int wave_inclusive_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);    // row_shr 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);    // lane 15 of rows 0, 2 to rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);    // lane 31 to rows 2, 3
    return v;
}

// 64 groups in a wave, a lane each: their rows, and the tiles of TILE rows up to
// and with each.
template <int TILE>
struct GroupLanes {
    int begin, end, incl;
    __device__ __forceinline__ void load(const GroupedArgs& a, int g0) {
        const int g = g0 + (threadIdx.x & 63);
        begin = end = 0;
        if (g < a.groups) group_range(a, g, &begin, &end);
        incl = wave_inclusive_sum((end - begin + TILE - 1) / TILE);
    }
    __device__ __forceinline__ int sum() const { return __builtin_amdgcn_readlane(incl, 63); }
    // The first lane whose sum is above `tiles`, which is below sum().
    __device__ __forceinline__ int past(int tiles) const { return __builtin_ctzll(__builtin_amdgcn_ballot_w64(incl > tiles)); }
    __device__ __forceinline__ int begin_of(int l) const { return __builtin_amdgcn_readlane(begin, l); }
    __device__ __forceinline__ int end_of(int l) const { return __builtin_amdgcn_readlane(end, l); }
    __device__ __forceinline__ int incl_of(int l) const { return __builtin_amdgcn_readlane(incl, l); }
};

// Block b's tile among the groups' tiles of TILE rows x tiles_n columns, in the
// order of the groups, within one as grouped_tile orders them, each XCD walking
// a contiguous run.  Every wave computes it for itself.  round > 0: the tiles past a
// whole number of rounds of `round`, if they are a quarter of one or less, go to
// four blocks each, which follow the others.
//
// Offsets that decrease let groups share rows, so that there may be more tiles
// than an int counts.  64 groups' sum is below 2^30 (the entry points' bound on
// row tiles, 2^23, for each); the total stops at kMostTiles, beyond any grid.  With
// that no number here overflows, and whatever the offsets hold, the tile lies in
// its group and the group in the matrix.
constexpr int kMostTiles = 1 << 28;
template <int TILE, typename Lanes = GroupLanes<TILE>>
__host__ __device__ __forceinline__ GroupRows locate_group_tile(const GroupedArgs& a, int b, int tiles_n, int group_m,
                                                                int round = 0) {
    Lanes lanes;
    int total = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
        lanes.load(a, g0);
        total += lanes.sum();
        if (total > kMostTiles) total = kMostTiles;
    }
    GroupRows r{0, 0, -1, 0, 0, -1};
    const int64_t tiles = (int64_t)total * tiles_n;
    int blocks = tiles < kMostTiles ? (int)tiles : kMostTiles;
    int rest = 0;
    if (round > 0) {
        rest = blocks % round;
        if (rest > round / 4) rest = 0;
        blocks -= rest;
    }
    if (b >= blocks + 4 * rest) return r;
    int logical;
    if (b < blocks) {
        logical = xcd_contiguous(b, blocks);
    } else {
        const int q = xcd_contiguous(b - blocks, 4 * rest);
        logical = blocks + q / 4;
        r.quarter = q % 4;
    }
    const int row = logical / tiles_n;                      // row tile if the tiles went row by row
    int before = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
        if (a.groups > 64) lanes.load(a, g0);
        if (row < before + lanes.sum()) {
            const int l = lanes.past(row - before);
            r.group = g0 + l;
            r.begin = lanes.begin_of(l);
            r.rows = lanes.end_of(l) - r.begin;
            const int tiles_m = (r.rows + TILE - 1) / TILE;
            const int first = before + lanes.incl_of(l) - tiles_m;
            const int local = logical - first * tiles_n;
            const int gsize = (group_m < tiles_m ? group_m : tiles_m) * tiles_n;
            const int q = local / gsize, first_m = q * group_m;
            const int gm = tiles_m - first_m < group_m ? tiles_m - first_m : group_m;
            const int in_q = local - q * gsize;
            r.tm = first_m + in_q % gm;
            r.tn = in_q / gm;
            return r;
        }
        before += lanes.sum();
    }
    return r;
}

// The group's share of a product and its epilogue.
__device__ __forceinline__ void enter_group(const GroupedArgs& a, const GroupRows& r, Gemm16Args* p, EpilogueArgs* e) {
    p->M = e->M = r.rows;
    p->A += (int64_t)r.begin * p->lda;
    p->B += r.group * a.stride_b;
    e->C = static_cast<char*>(e->C) + (e->c_type == 2 ? 4 : 2) * (r.begin * e->ldc);
    if (e->residual != nullptr)
        e->residual = static_cast<const char*>(e->residual) + (e->c_type == 2 ? 4 : 2) * (r.begin * e->ldr);
    if (e->preact != nullptr) e->preact = static_cast<char*>(e->preact) + 2 * (r.begin * e->ldz);
    if (e->bias != nullptr)
        e->bias = static_cast<const char*>(e->bias) + (e->bias_type == 2 ? 4 : 2) * (r.group * a.ld_bias);
}

// The weights' gradient: block b's group and tile.  The tiles of a group are
// shared by the XCDs: groups differ in their rows, so whole groups to an XCD
// would not balance.
__device__ __forceinline__ GroupRows locate_grad_tile(const GroupedArgs& a, int b, int tiles_m, int tiles_n, int group_m) {
    const int tiles = tiles_m * tiles_n;
    GroupRows r;
    r.group = b / tiles;
    grouped_tile(b - r.group * tiles, tiles_m, tiles_n, group_m, &r.tm, &r.tn);
    int end;
    group_range(a, r.group, &r.begin, &end);
    r.rows = end - r.begin;
    return r;
}
__device__ __forceinline__ void enter_grad_group(const GroupedArgs& a, const GroupRows& r, Gemm16Args* p, EpilogueArgs* e) {
    p->A += (int64_t)r.begin * p->lda;
    p->B += (int64_t)r.begin * p->ldb;
    p->K = r.rows;
    e->C = static_cast<char*>(e->C) + (e->c_type == 2 ? 4 : 2) * (r.group * a.stride_b);
}

}  // namespace
#endif

// Tiles of bm x bn (grouped_shared.hip): 128 x 256, 128 x 128, 64 x 256, 64 x
// 128; the gradient's of 128 rows.  direct: the operands are copied straight into
// LDS, for bases on 4 bytes, even leading dimensions and strides, even widths of
// the factors that are not k-contiguous, an even K otherwise (the gradient: any
// rows), and operands within the copies' offsets; the caller
// checks.  Otherwise any problem, on 128 columns.  K split over blocks (k_share a
// multiple of 32 below K; splits above 1): each stores its sums as a plane of
// binary32 values, `plane` of them after the one before, e then being the first
// plane.
hipError_t launch_grouped_shared(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                                 int format, int op_b, bool direct, int bm, int bn, int k_share, int64_t plane);
hipError_t launch_grouped_grad_shared(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                                      int format, bool direct, int bn, int splits, int64_t plane);

// p: A, B, N, K and their leading dimensions (M is not used); e: M is not used.
int64_t grouped_workspace(const GroupedArgs& a, const Gemm16Args& p, int op_b);
hipError_t launch_grouped(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s, int format,
                          int op_b, void* workspace);
// The weights' gradient: p.M x p.N per group from A (rows x M) and B (rows x N), both
// as stored; e: C, its type and leading dimension.
int64_t grouped_grad_workspace(const GroupedArgs& a, const Gemm16Args& p);
hipError_t launch_grouped_grad(const GroupedArgs& a, const Gemm16Args& p, const EpilogueArgs& e, hipStream_t s,
                               int format, void* workspace);
// dZ = dY act'(Z) over the groups' rows, and the groups' column sums (e.bias_grad: groups x N).
int64_t grouped_activation_workspace(int64_t rows, int64_t groups, int64_t N);
hipError_t launch_grouped_activation(const GroupedArgs& a, const EpilogueArgs& e, const uint16_t* dY, int64_t ld,
                                     float* partials, hipStream_t s);

}  // namespace gemmf32
