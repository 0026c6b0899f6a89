// grouped_plan.h -- the layer whose rows belong to groups: which tile and how many
// blocks along K a call takes, by estimated times (host only; not part of the
// public interface).
#pragma once

#include "grouped_kernels.h"

#include <math.h>

namespace gemmf32 {

namespace {

// A factor of `rows` rows whose copies' 32-bit offsets hold, a tile's
// overhang included.
bool offsets_hold(int64_t rows, int64_t ld) { return ld < (1ll << 30) / (rows + 256); }
bool even_base(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Whether the operands can be copied straight into LDS.
bool direct_fits(const GroupedArgs& a, const Gemm16Args& p, int op_b) {
    return p.K > 0 && p.K % 2 == 0 && p.lda % 2 == 0 && p.ldb % 2 == 0 && a.stride_b % 2 == 0 && (op_b || p.N % 2 == 0) &&
           even_base(p.A) && even_base(p.B) && offsets_hold(256, p.lda) && offsets_hold(op_b ? p.N : p.K, p.ldb);
}
bool direct_grad_fits(const GroupedArgs& a, const Gemm16Args& p) {
    return p.lda % 2 == 0 && p.ldb % 2 == 0 && p.M % 2 == 0 && p.N % 2 == 0 && even_base(p.A) && even_base(p.B) &&
           offsets_hold(a.rows, p.lda) && offsets_hold(a.rows, p.ldb);
}

// Groups that have a row, if every row chooses one with the same chance.
double used_groups(int groups, int rows) { return groups * (1.0 - pow(1.0 - 1.0 / groups, rows)); }

// Row tiles that the groups make on average: each group leaves half a tile.
double expected_row_tiles(int groups, int rows, int tile) {
    if (groups == 1) return ceil_div(rows, tile);
    const double used = used_groups(groups, rows);
    return used * fmax(1.0, rows / used / tile + 0.5);
}

// Estimated time of `tiles` tiles of `phases` steps of 32 k, in us.  A block
// alone on a CU takes `alone` per phase, which is the memory's latency over the
// stages in flight; with `slots` of them on the chip (two to four to a CU) a
// round of them takes `full` per phase; and `fixed` for start and epilogue.  How
// many rounds the groups' rows make is not known here: past one, half a round
// more for the last.  (4096^3 in one group: 121 us on 128 x 256 tiles, 157 on 128
// x 128, 157 on 64 x 256, 185 on 64 x 128; 1024 x 1024 x 1024 in 16 groups: 28 /
// 19 / 19 / 15.)
struct Shape {
    int bm, bn, slots;
    double alone, full, fixed;
};
constexpr Shape kShapes[] = {
    {128, 256, 512, 0.45, 0.84, 13.5}, {128, 128, 768, 0.43, 0.875, 5.1}, {64, 256, 512, 0.45, 0.575, 5.0},
    {64, 128, 768, 0.305, 0.50, 5.0}};
// The kernels through registers, by the weight's orientation (whole runs of k take
// fewer registers and more time), and the gradient's: figures that choose best among
// the tiles and splits timed at 44, 44 and 34 odd shapes, 1.6, 1.8 and 2.1 % above
// the fastest on average, where those of the direct kernels choose 1.9, 3.7 and 2.8 %
// above.  (2048 x 2047 x 4097 in one group with N x K weights 68 us on 128 x 128 tiles
// against 85 on 64 x 128.)
constexpr Shape kStaged[2][2] = {{{128, 128, 512, 0.44, 0.675, 11.3}, {64, 128, 1024, 0.26, 0.97, 7.2}},
                                 {{128, 128, 768, 0.36, 1.33, 6.9}, {64, 128, 1024, 0.285, 1.105, 3.3}}};
constexpr Shape kStagedGrad = {128, 128, 512, 0.535, 1.06, 7.1};
double tiles_time(const Shape& c, double tiles, double phases) {
    if (tiles > c.slots) return (tiles / c.slots + 0.5) * (c.full * phases + c.fixed);
    const double busy = fmax(0.0, (tiles - 256.0) / (c.slots - 256.0));
    return (c.alone + (c.full - c.alone) * busy) * phases + c.fixed;
}

// The pass over `splits` planes of `values`, from 4 us, at 3 TB/s.
double pass_time(int splits, double values) { return 4.0 + 4.0 * splits * values / 3e6; }

struct Plan {
    bool direct;
    int bm, bn;
    int splits, k_share;               // blocks along K; k of each
    int64_t bytes;                     // of planes, if split
};

Plan make_plan(const GroupedArgs& a, const Gemm16Args& p, int op_b) {
    Plan q{};
    q.splits = 1;
    q.k_share = p.K;
    q.direct = direct_fits(a, p, op_b);
    if (p.K == 0) {                    // the epilogue alone
        q.bm = 64;
        q.bn = 128;
        q.k_share = 1;
        return q;
    }
    const int phases = ceil_div(p.K, 32);
    double least = 1e30;
    const Shape* const shapes = q.direct ? kShapes : kStaged[op_b != 0];
    for (const Shape* s = shapes; s != shapes + (q.direct ? 4 : 2); ++s) {
        const Shape& c = *s;
        const double tiles = expected_row_tiles(a.groups, a.rows, c.bm) * ceil_div(p.N, c.bn);
        for (int splits = 1; splits <= 16 && (splits == 1 || (tiles * splits <= c.slots && phases >= 8 * splits)); splits *= 2) {
            const double t = tiles_time(c, tiles * splits, (double)phases / splits) +
                             (splits > 1 ? pass_time(splits, (double)a.rows * p.N) : 0.0);
            if (t < least) {
                least = t;
                q.bm = c.bm;
                q.bn = c.bn;
                q.k_share = splits > 1 ? 32 * ceil_div(phases, splits) : p.K;
                q.splits = ceil_div(p.K, q.k_share);
            }
        }
    }
    if (q.splits > 1) q.bytes = 4 * (int64_t)q.splits * a.rows * p.N;
    return q;
}

// The weights' gradient: 128 x 256 tiles for groups of 384 rows and more that make
// about one whole round of the 512 on the chip or two and more (16384 x 2048 x 4096
// over 2 groups 249 us against 294 on 128 x 128, 8192 x 2048 x 4096 over 16 147
// against 161), else 128 x 128, which store sooner (4096 x 1024 x 2048 over 64 63
// us against 70, 2000 x 1000 x 1000 over 4 15 against 20); few tiles with long
// groups split the rows.
Plan make_grad_plan(const GroupedArgs& a, const Gemm16Args& p) {
    Plan q{};
    q.splits = 1;
    q.direct = direct_grad_fits(a, p);
    q.bm = 128;
    const int64_t wide = (int64_t)a.groups * ceil_div(p.M, 128) * ceil_div(p.N, 256);
    const double rows = a.rows / used_groups(a.groups, a.rows > 0 ? a.rows : 1);
    q.bn = q.direct && rows >= 384 && ((wide >= 448 && wide <= 512) || wide >= 1024) ? 256 : 128;
    if (q.bn == 256) return q;
    const double tiles = (double)a.groups * ceil_div(p.M, 128) * ceil_div(p.N, 128);
    const double phases = ceil(rows / 32.0);
    double least = 1e30;
    const Shape& c = q.direct ? kShapes[1] : kStagedGrad;
    for (int splits = 1; splits <= 32 && (splits == 1 || (tiles * splits <= c.slots && phases >= 8 * splits)); splits *= 2) {
        const double t = tiles_time(c, tiles * splits, phases / splits) +
                         (splits > 1 ? pass_time(splits, (double)a.groups * p.M * p.N) : 0.0);
        if (t < least) {
            least = t;
            q.splits = splits;
        }
    }
    if (q.splits > 1) q.bytes = 4 * (int64_t)q.splits * a.groups * p.M * p.N;
    return q;
}

}  // namespace

}  // namespace gemmf32
