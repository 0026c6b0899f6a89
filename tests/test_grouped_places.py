"""Where the blocks of the grouped layer's kernels work, on the host: in range,
every place once."""
import ctypes

import pytest

from host_code import compile_host

SOURCE = r"""
#include "grouped_kernels.h"
using namespace gemmf32;
extern "C" void share_of(int rows, int splits, int i, long long* out) {
    const RowShare s = row_share(rows, splits, i);
    out[0] = s.first;
    out[1] = s.rows;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return compile_host(tmp_path_factory.mktemp("host"), SOURCE)


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
