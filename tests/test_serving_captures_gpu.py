"""Serving-step calls in captured graphs whose streams fork and join, after copies and fills, and in two graphs that
share one workspace, replayed one after the other."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_serving_gpu import PLANS, check_rows, err_word, i32, outputs, q4_pool, queries, rope_case, workspace

pytestmark = pytest.mark.gpu
BK = 128


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def test_calls_after_forks_joins_and_fills(msa):
    """Each call comes after two streams' joined work, a fill or a copy, and a join follows it."""
    L, n, pt, free, count, N, pool = PLANS["edges"]()
    want = ref.plan(L, n, pt, free, count, N, pool)
    src = {"L": i32(L), "n": i32(n), "pt": i32(pt), "free": i32(free), "count": i32([count])}
    t = {k: torch.zeros_like(v) for k, v in src.items()}
    o, err = msa.plan_buffers(len(L), N, "cuda"), err_word()
    Q, K, V, wq, wk, _, f = rope_case(N, 12, 2, 128, 128, 31)
    Qo, Ko = torch.zeros(N, 12, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, 2, 128, dtype=torch.bfloat16, device="cuda")
    cache = msa.q4_cache(pool, 2, "cuda")
    B = len(L)
    O, LSE, ws = torch.zeros(B, 12, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, 12, device="cuda"), workspace(msa, B, 2)
    Kx, Vx = (torch.zeros(pool, 2, BK, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, pages = queries(B, 12, 32), torch.arange(pool, dtype=torch.int32, device="cuda")
    rows, heads = i32(np.repeat(want["seq_pt"], 2, 0)), want["seq_len_out"]
    rn, rl = i32(np.repeat(-(-heads // BK), 2)), i32(np.repeat(np.where(heads > 0, (heads - 1) % BK + 1, 0), 2))
    So, Sl, ws2 = torch.zeros_like(O), torch.zeros_like(LSE), workspace(msa, B, 2)

    def step(main, side):
        for k, v in src.items():
            t[k].copy_(v)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for x in cache[:4]:
                x.zero_()
        msa.msa_plan_step(t["L"], t["n"], t["pt"], t["free"], t["count"], *o.values(), num_pages=pool, dev_err=err)
        main.wait_stream(side)                                   # a call after a join of two streams
        msa.msa_qk_norm_rope(Q, K, o["tok_pos"], f, Qo, Ko, q_weight=wq, k_weight=wk, dev_err=err)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            O.fill_(3.0)
        msa.msa_cache_append_q4(Ko, V, o["tok_slot"], cache, dev_err=err)
        main.wait_stream(side)
        side.wait_stream(main)
        with torch.cuda.stream(side):                            # two branches of this library's calls
            msa.msa_cache_expand_q4(cache, pages, Kx, Vx, dev_err=err)
            msa.msa_sparse_attn_decode_q4(q, cache, rows, rn, rl, So, Sl, ws2, dev_err=err)          # (clears its scratch)
        msa.msa_dense_attn_decode_q4(q, cache, t["pt"], o["seq_len_out"], O, LSE, ws, dev_err=err, scratch_zeroed=True)
        main.wait_stream(side)
        msa.msa_release_pages(o["seq_len_out"], t["n"], t["pt"], t["free"], o["free_count_out"], o["seq_len_out"], o["free_count_out"],
                              num_pages=pool, dev_err=err)

    def check():
        torch.cuda.synchronize()
        assert int(err) == 0
        for k in ("tok_slot", "tok_pos", "tok_seq", "cu"):
            assert np.array_equal(o[k].cpu(), want[k]), k
        assert np.array_equal(t["pt"].cpu(), want["seq_pt"])
        for out, lse in ((O, LSE), (So, Sl)):
            check_rows(q, out, lse, lambda b, g: want["seq_pt"][b, :-(-heads[b] // BK)], lambda b, g: heads[b], cache)
        back = ref.release(want["seq_len_out"], n, want["seq_pt"], np.array(free), want["free_count_out"])
        assert np.array_equal(o["seq_len_out"].cpu(), back["seq_len_out"]) and int(o["free_count_out"]) == back["free_count_out"]

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        step(main, side)
    check()
    keep = [x.clone() for x in (O, LSE, So, Sl, Qo, Ko, Kx, Vx)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        step(main, side)
    for x in (O, LSE, So, Sl, Qo, Ko, Kx, Vx, *o.values()):
        x.zero_()
    for _ in range(3):
        graph.replay()
    check()
    for a, b in zip(keep, (O, LSE, So, Sl, Qo, Ko, Kx, Vx)):
        assert torch.equal(a, b)


def test_two_graphs_share_a_workspace(msa):
    """A dense and a sparse attention of other sizes captured over one zero-filled workspace, replayed in turn, with
    calls outside a graph between them."""
    c, ws = q4_pool(msa, 40, 2, 33), workspace(msa, 70, 2)
    pt, L = i32(np.arange(40)[None].repeat(3, 0)), i32([40 * BK, 5, 3000])
    rows = i32(np.arange(140 * 16).reshape(140, 16) % 40)
    n, last = i32(np.full(140, 16)), i32(np.full(140, 77))
    Qd, Qs = queries(3, 12, 34), queries(70, 12, 35)
    want = outputs(3, 12), outputs(70, 12)
    msa.msa_dense_attn_decode_q4(Qd, c, pt, L, *want[0], workspace(msa, 3, 2))
    msa.msa_sparse_attn_decode_q4(Qs, c, rows, n, last, *want[1], workspace(msa, 70, 2))
    got = outputs(3, 12), outputs(70, 12)
    calls = [lambda: msa.msa_dense_attn_decode_q4(Qd, c, pt, L, *got[0], ws, scratch_zeroed=True),
             lambda: msa.msa_sparse_attn_decode_q4(Qs, c, rows, n, last, *got[1], ws, scratch_zeroed=True)]
    for f in calls:
        f()
    torch.cuda.synchronize()
    graphs = []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for order in ((0, 1), (1, 0), (1, 1), (0, 0)):
        for x in (*got[0], *got[1]):
            x.fill_(9.0)
        for i in order:
            graphs[i].replay()
            calls[1 - i]()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
