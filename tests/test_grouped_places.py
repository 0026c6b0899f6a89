"""Where the blocks of the grouped layer's kernels work, on the host: in range,
every place once."""
import ctypes
import random

import pytest

from host_code import compile_host

SOURCE = r"""
#include "grouped_kernels.h"
using namespace gemmf32;

#include <map>
#include <tuple>

// 64 groups at a time as a wave holds them.
template <int TILE>
struct HostLanes {
    int begin[64], end[64], incl[64];
    void load(const GroupedArgs& a, int g0) {
        int sum = 0;
        for (int l = 0; l < 64; ++l) {
            begin[l] = end[l] = 0;
            if (g0 + l < a.groups) group_range(a, g0 + l, &begin[l], &end[l]);
            sum += (end[l] - begin[l] + TILE - 1) / TILE;
            incl[l] = sum;
        }
    }
    int sum() const { return incl[63]; }
    int past(int tiles) const {
        for (int l = 0; l < 64; ++l)
            if (incl[l] > tiles) return l;
        return 64;                                          // of an empty mask
    }
    int begin_of(int l) const { return begin[l & 63]; }
    int end_of(int l) const { return end[l & 63]; }
    int incl_of(int l) const { return incl[l & 63]; }
};

// Every step-th block of the grid that the launcher starts: 1 + the number of the
// first whose tile lies outside its group or whose group lies outside the
// matrix, 0 if none.  once: also, over all blocks, every tile once or its quarters.
template <int TILE>
long long places(const GroupedArgs& a, long long tiles_n, int group_m, int round, long long step, bool once) {
    long long blocks = grouped_row_tiles(a.rows, a.groups, TILE) * tiles_n;
    if (round > 0) blocks += 3 * std::min<long long>(blocks, round / 4);
    std::map<std::tuple<int, int, int>, int> seen;
    for (long long b = 0; b < blocks; b += step) {
        const GroupRows r = locate_group_tile<TILE, HostLanes<TILE>>(a, (int)b, (int)tiles_n, group_m, round);
        if (r.rows < 0) continue;
        const bool in = r.group >= 0 && r.group < a.groups && r.begin >= 0 && (long long)r.begin + r.rows <= a.rows &&
                        r.tm >= 0 && (long long)r.tm * TILE < r.rows && r.tn >= 0 && r.tn < tiles_n && r.quarter >= -1 &&
                        r.quarter < 4 && (round > 0 || r.quarter < 0);
        if (!in) return 1 + b;
        if (once) {
            int& parts = seen[{r.group, r.tm, r.tn}];
            const int part = r.quarter < 0 ? 15 : 1 << r.quarter;
            if (parts & part) return 1 + b;
            parts |= part;
        }
    }
    if (once) {
        long long tiles = 0;
        for (int g = 0; g < a.groups; ++g) tiles += (a.offsets[g + 1] - a.offsets[g] + TILE - 1) / TILE * tiles_n;
        if ((long long)seen.size() != tiles) return -1;
        for (const auto& s : seen)
            if (s.second != 15) return -2;
    }
    return 0;
}
extern "C" long long places_of(int tile, int groups, const int* offsets, int rows, long long tiles_n, int group_m,
                               int round, long long step, int once) {
    const GroupedArgs a{groups, offsets, rows, 0, 0};
    if (tile == 16) return places<16>(a, tiles_n, group_m, round, step, once);
    if (tile == 64) return places<64>(a, tiles_n, group_m, round, step, once);
    return places<128>(a, tiles_n, group_m, round, step, once);
}

extern "C" void share_of(int rows, int splits, int i, long long* out) {
    const RowShare s = row_share(rows, splits, i);
    out[0] = s.first;
    out[1] = s.rows;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    lib = compile_host(tmp_path_factory.mktemp("host"), SOURCE)
    lib.places_of.restype = ctypes.c_longlong
    lib.places_of.argtypes = [ctypes.c_int] * 2 + [ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_int,
                                                   ctypes.c_int, ctypes.c_longlong, ctypes.c_int]
    return lib


# around every power of two, and all the way up to the rows that the entry point takes
ROWS = sorted({n for b in range(32) for n in (2 ** b - 1, 2 ** b, 2 ** b + 1, 3 * 2 ** b + 5) if 0 < n < 2 ** 31} |
              {0, 2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 31, 2 ** 31 - 32, 2 ** 31 - 33, 2 ** 31 - 1023, 2 ** 31 - 1024, 2 ** 31 - 1025})


@pytest.mark.parametrize("splits", [1, 2, 4, 8, 16, 32])
def test_shares_of_rows(host, splits):
    """Shares follow one another, in whole steps of 32 rows but for the last, and
    together are all rows."""
    out = (ctypes.c_longlong * 2)()
    for rows in ROWS:
        at = 0
        for i in range(splits):
            host.share_of(rows, splits, i, out)
            first, count = out[0], out[1]
            assert 0 <= count and first == at, (rows, i)
            assert count % 32 == 0 or first + count == rows, (rows, i)
            at += count
        assert at == rows, rows


def places(host, tile, offsets, rows, tiles_n, group_m, round_=0, step=1, once=False):
    held = (ctypes.c_int32 * len(offsets))(*offsets)
    return host.places_of(tile, len(offsets) - 1, held, rows, tiles_n, group_m, round_, step, once)


# tile, its order within a group and the rounds whose rest is divided, as the kernels take them
FORMS = [(16, 1, 0), (64, 16, 0), (64, 1 << 20, 0), (128, 8, 0), (128, 8, 512), (128, 8, 12)]


@pytest.mark.parametrize("tile,group_m,round_", FORMS, ids=str)
def test_every_tile_once(host, tile, group_m, round_):
    rng = random.Random(tile + round_)
    for counts in ([1], [0], [0, 0, 3, 0], [64] * 64, [1] * 65, [127, 0, 129, 128] * 40, [5000], [0] * 200 + [300],
                   [rng.randrange(400) for _ in range(130)], [rng.randrange(3000) for _ in range(9)]):
        for lead, tail in ((0, 0), (7, 100)):
            offsets = [lead]
            for c in counts:
                offsets.append(offsets[-1] + c)
            for tiles_n in (1, 2, 5, 16):
                assert places(host, tile, offsets, offsets[-1] + tail, tiles_n, group_m, round_, once=True) == 0, counts


@pytest.mark.parametrize("tile,group_m,round_", FORMS, ids=str)
def test_offsets_of_any_content(host, tile, group_m, round_):
    """Offsets that decrease, are negative or pass the rows: no tile outside."""
    rng = random.Random(7 * tile + round_)
    low, high = -2 ** 31, 2 ** 31 - 1
    for rows in (1, 63, 64, 1000, 4097):
        for groups in (1, 3, 64, 65, 300):
            for kind in range(5):
                offsets = [rng.choice(([0, rows], [low, high], [rows, 0, high, low, rows // 2], [rng.randint(low, high)],
                                       [rng.randint(-rows, 2 * rows)])[kind]) for _ in range(groups + 1)]
                for tiles_n in (1, 3, 40):
                    assert places(host, tile, offsets, rows, tiles_n, group_m, round_) == 0, (rows, offsets)


# the most rows, columns and groups that the entry points take: the row tiles of all groups pass 2^31
@pytest.mark.parametrize("tile,group_m,round_", [f for f in FORMS if f[0] != 16], ids=str)
@pytest.mark.parametrize("groups,rows,tiles_n", [(65535, 500_000_000, 1), (65535, 2_000_000, 80), (4000, 2 ** 20, 255),
                                                 (65535, 100, 1000), (1, 64 * ((1 << 23) - 1), 1), (9, 64 * 100, 80000)])
def test_offsets_that_decrease_over_many_rows(host, tile, group_m, round_, groups, rows, tiles_n):
    blocks = -(-(rows + min(groups, rows) * (tile - 1)) // tile) * tiles_n
    for offsets in ([0 if g % 2 else rows for g in range(groups + 1)], [rows if g % 2 else 0 for g in range(groups + 1)],
                    [rows - g if g % 2 else g for g in range(groups + 1)]):
        assert places(host, tile, offsets, rows, tiles_n, group_m, round_, step=max(1, blocks // 200)) == 0
