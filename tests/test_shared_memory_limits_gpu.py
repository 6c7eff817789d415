"""Calls of one kernel from two threads, with batches whose tables need different amounts of shared memory: each is served, whatever
the other asks for.  (The limit of a kernel's shared memory belongs to the kernel, not to a launch.)"""
import ctypes as C
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
BK, MOST = 128, 4096


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def i32(*shape, value=0):
    return torch.full(shape, value, dtype=torch.int32, device="cuda")


def fork(msa, B):
    """B forks that are all padding: the call reads and writes its tables and changes nothing."""
    src, L, pt, free, n, shares = i32(B, value=-1), i32(B), i32(B, 2), i32(8), i32(1), i32(8)
    out = i32(B), i32(B)
    return lambda s: msa.msa_fork_requests(src, src, L, pt, free, n, shares, L, pt, n, shares, *out, stream=s)


def plan(msa, B):
    """B requests that bring no token."""
    L, pt, free, n, cu = i32(B), i32(B, 2), i32(8), i32(1), i32(B + 1)
    new, seq, pos, slot = i32(B), i32(16), i32(16), torch.zeros(16, dtype=torch.int64, device="cuda")
    return lambda s: msa.msa_plan_step(L, new, pt, free, n, L, n, cu, slot, pos, seq, num_pages=8, stream=s)


def index(msa, B):
    """The index score and selection of B sequences of one token, by the C entry point itself (Python takes longer to marshal it)."""
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    keep = [torch.ones(B, 1, 4, 64, **bf16), torch.ones(B, 1, 4, device="cuda"), torch.ones(2, 1, BK, 64, **bf16),
            torch.empty(B, 1, 4, device="cuda"), i32(B, 1), i32(B, value=1), i32(B, 1, 4), i32(B, 1), i32(B)]
    from block_sparse_attention_02_gb300 import _abi
    a = _abi.IndexArgs()
    a.mode, a.B, a.Hkv, a.HI, a.dI, a.Bk, a.num_pages, a.max_pages, a.nb_stride, a.k = msa.MSA_MODE_DECODE, B, 1, 4, 64, BK, 2, 1, 4, 4
    a.q_idx, a.w, a.k_idx, a.C, a.seq_pt, a.seq_len, a.sel, a.count, a.row_scratch = [t.data_ptr() for t in keep]
    a.q_idx_stride[:], a.w_stride[:], a.k_idx_stride[:], a.C_stride[:] = [256, 256, 64, 0], [4, 4, 0], [BK * 64, BK * 64, 64], [4, 4, 0]
    f = msa.lib().msa_index_score

    def call(s, keep=keep):
        _abi.check(f(C.byref(a), s.cuda_stream), "msa_index_score")
    return call


@pytest.mark.parametrize("make,small", [(fork, 2600), (plan, 3500), (index, 8)])
def test_two_threads(msa, make, small):
    large = 1024 if make is index else MOST
    calls, wrong = [make(msa, large), make(msa, small)], []
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(call, s):
        try:
            for i in range(4000 if make is not index else 20000):
                call(s)
                if i % 200 == 0:
                    s.synchronize()
        except Exception as e:       # noqa: BLE001 (a thread's own exception would not fail the test)
            wrong.append(str(e))
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong[0]
