"""Where the rotated queries of a rotating append may go (no GPU): what overlaps
no row of q, k or v is taken, also between their rows."""

import pytest

from test_host_fp4_beam import _rope
from test_host_paged import FAKE, B  # noqa: F401


@pytest.mark.parametrize("dtype, es", [(0, 4), (1, 2)])
def test_queries_may_leave_between_the_rows_of_the_projection(B, dtype, es):
    # rows of [q 4096 | k 1024 | v 1024 | 4096 for the rotated queries]
    at = dict(q=FAKE, k=FAKE + 4096 * es, v=FAKE + 5120 * es, ld=10240, dtype=dtype, ws=0)
    out = FAKE + 6144 * es
    assert _rope(B, **at, out=out, old=10240) == -4           # all in order but the workspace
    assert _rope(B, **at, out=FAKE, old=10240) == -4          # in place, as before
    # rows before q, of the same buffer
    assert _rope(B, **{**at, "q": out, "k": out + 4096 * es, "v": out + 5120 * es, "ld": 12288}, out=FAKE, old=12288) == -4
    # over the end of v, into the next row's q, at another distance
    assert _rope(B, **at, out=out - 16, old=10240) == -1
    assert _rope(B, **at, out=out + 16, old=10240) == -1
    assert _rope(B, **at, out=out, old=10240 + 16 // es) == -1
    # a row later, or one that begins inside the rows
    assert _rope(B, **at, out=out + 10240 * es, old=10240) == -4
    assert _rope(B, **at, out=FAKE + 10240 * es, old=10240) == -1
