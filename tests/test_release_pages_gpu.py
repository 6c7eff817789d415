"""Pages that go back on the stack: ids outside the pool and bad stack heights."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_serving_gpu import err_word, i32

pytestmark = pytest.mark.gpu
BK = 128


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def release(msa, L, done, pt, free, count, in_place=False, **kw):
    t = i32(L), i32(done), i32(pt), i32(free), i32([count])
    out, cnt, e = (t[0], t[4], err_word()) if in_place else (torch.full_like(t[0], -7), i32([-1]), err_word())
    msa.msa_release_pages(*t, out, cnt, dev_err=e, **kw)
    return out.cpu().numpy(), int(cnt), t[3].cpu().numpy(), int(e)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [1, 9, 900])
def test_ids_outside_the_pool_are_named(msa, B, in_place):
    """They go back as they are, and the error word says so; ids that stay in their tables are nobody's concern."""
    r, mp = np.random.default_rng(B), 6
    pool = B * mp
    L = r.integers(2 * BK + 1, mp * BK + 1, B)
    done = (r.random(B) < 0.5).astype(np.int64)
    done[0] = 1
    pt = r.permutation(pool).reshape(B, mp)
    free = np.full(pool + 3, -5)

    def check(num_pages, bad):
        want = ref.release(L, done, pt, free, 3)
        kw = {} if num_pages is None else {"num_pages": num_pages}
        out, cnt, stack, e = release(msa, L, done, pt, free, 3, in_place, **kw)
        assert np.array_equal(out, want["seq_len_out"]) and cnt == want["free_count_out"] and np.array_equal(stack, want["free_pages"])
        assert e == want["err"] | (msa.MSA_DEVERR_BAD_PAGE if bad else 0)

    check(None, False), check(pool, False)
    if B > 1:
        kept = int(np.flatnonzero(done == 0)[0]) if (done == 0).any() else None
        if kept is not None:
            pt[kept, 0] = -3                                     # not returned
            check(pool, False)
    L[0] = 2 * BK
    pt[0, 2] = -1                                                # past the request's pages
    check(pool, False)
    was = pt[0, 1]
    pt[0, 1] = -1
    check(None, True), check(pool, True)
    pt[0, 1] = pool
    check(None, False), check(pool, True), check(pool + 1, False)
    pt[0, 1] = was
    check(pool, False)


@pytest.mark.parametrize("in_place", [False, True])
def test_stack_heights_outside_the_stack(msa, in_place):
    """Below 0 counts as 0, past the end as full (every page is dropped); both are named."""
    r = np.random.default_rng(3)
    L, done, pt = np.array([300, 128, 0, 700]), np.array([1, 0, 1, 1]), r.permutation(24).reshape(4, 6)
    for cap in (40, 5):
        free = r.permutation(cap)
        for count in (-3, cap + 5, cap, 0):
            want = ref.release(L, done, pt, free, count)
            out, cnt, stack, e = release(msa, L, done, pt, free, count, in_place, num_pages=24)
            assert np.array_equal(out, want["seq_len_out"]) and cnt == want["free_count_out"] and np.array_equal(stack, want["free_pages"])
            assert e == want["err"]
