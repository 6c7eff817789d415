"""Forks of a request whose partly filled page's id, or whose own new page's, lies outside the pool: msa_copy_pages could only
leave such a pair out, so the fork says so (the rest as the serial definition has it)."""
import numpy as np
import pytest

import cache_ref as ref
from test_shared_pages_gpu import BK, msa, requests, run_fork  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, -(1 << 31), "pool", (1 << 31) - 1])
@pytest.mark.parametrize("where", ["table", "stack"])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_of_a_bad_partial_page(msa, bad, where, in_place):  # noqa: F811
    L, pt, free, count, shares = requests(1, [300, 0, 256, 0, 0, 130], 6, 4)
    bad = len(shares) if bad == "pool" else bad
    if where == "table":
        pt[0, 2] = bad                                     # of 300 tokens the last 44
    else:
        free[count - 1] = bad                              # the page that the first fork gets
    want = ref.fork([0, 2, 5], [1, 3, 4], L, pt, free, count, shares)
    got = run_fork(msa, [0, 2, 5], [1, 3, 4], L, pt, free, count, shares, in_place)
    for k, v in want.items():
        if k != "err":
            assert np.array_equal(got[k], v), k
    assert got["err"] == msa.MSA_DEVERR_BAD_PAGE
    # full pages alone: the pages behind them are not looked at
    pt[2, 2], free[count - 1] = -1, -1
    assert run_fork(msa, [2], [3], L, pt, free, count, shares, in_place)["err"] == 0
