"""The calls of the C++ binding beside other Python threads."""
import threading
import time

import numpy as np
import pytest
import torch

import serving_ref as ref
from test_serving_gpu import PLANS, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def test_a_launch_that_waits_holds_no_other_thread(msa):
    """A stream's queue filled behind a kernel of about a second: the thread that fills it waits in a launch, another
    one goes on."""
    c = PLANS["edges"]()
    want = ref.plan(*c)
    t = [i32(x) for x in (c[0], c[1], c[2], c[3], [c[4]])]
    o = msa.plan_buffers(len(c[0]), c[5], "cuda")
    msa.msa_plan_step(*t, *o.values(), num_pages=c[6])
    torch.cuda.synchronize()
    spent = []

    def fill():
        start = time.perf_counter()
        torch.cuda._sleep(2_000_000_000)
        for _ in range(8000):
            msa.msa_plan_step(*t, *o.values(), num_pages=c[6])
        spent.append(time.perf_counter() - start)

    worker = threading.Thread(target=fill)
    worker.start()
    last, longest = time.perf_counter(), 0.0
    while worker.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        last, longest = now, max(longest, now - last)
    worker.join()
    torch.cuda.synchronize()
    assert np.array_equal(o["tok_slot"].cpu(), want["tok_slot"])
    if spent[0] < 0.5:
        pytest.skip("the queue took every launch")
    assert longest < 0.25, f"stopped for {longest:.2f} s of {spent[0]:.2f} s"
