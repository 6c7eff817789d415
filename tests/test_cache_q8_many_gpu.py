"""The 8-bit cache where there is much to do at once: stores of 600 to 1,024 tokens whose CTAs take several heads, sparse rows past
those that run together, and a page copy beside other calls."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import test_cache_q8_gpu as base
from test_cache_q8_gpu import msa  # noqa: F401

pytestmark = pytest.mark.gpu
BK, D = 128, 128


def slots_of(g, runs, pages):
    """Runs (first row, length) in pages of their own, in a random order of pages."""
    order, at = torch.randperm(pages, generator=g).tolist(), []
    for page, (t, n) in zip(order, runs):
        at += [page * BK + t + i for i in range(n)]
    return at


def check_store(msa, calls, pages, H, seed):  # noqa: F811
    """Every call's (K, V, slots) into pages of arbitrary codes and scales, against the serial definition, byte for byte."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = msa.q8_cache(pages, H, "cuda")
    for codes, scales in ((cache.K_codes, cache.K_scales), (cache.V_codes, cache.V_scales)):
        codes.copy_(torch.randint(0, 0x7F, codes.shape, generator=g, device="cuda"))
        scales.copy_(torch.randint(110, 125, scales.shape, generator=g, device="cuda"))
    want = [(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((cache.K_codes, cache.K_scales), (cache.V_codes, cache.V_scales))]
    for K, V, slots in calls:
        e = base.err_word()
        msa.msa_cache_append_q8(K.cuda(), V.cuda(), base.dev(slots, torch.int64), cache, dev_err=e)
        assert int(e.item()) == 0
        for (codes, scales), x in zip(want, (K, V)):
            ref.store(codes, scales, x.double().numpy(), np.asarray(slots))
        for (codes, scales), c, s in zip(want, (cache.K_codes, cache.V_codes), (cache.K_scales, cache.V_scales)):
            assert np.array_equal(s.cpu().numpy(), scales)
            assert np.array_equal(c.cpu().numpy(), codes)


# (tokens, heads): 2 * (tokens / 16) * heads passes four CTAs on each of 152 SMs, so a CTA has 2, 2 or 4 heads (the last one 1)
@pytest.mark.parametrize("N,H", [(640, 8), (1024, 8), (1000, 13)])
def test_decoded_tokens_whose_blocks_grow(msa, N, H):  # noqa: F811
    """Every token to a page of its own; then a second, larger one behind it, so that every block is rounded again."""
    g = torch.Generator().manual_seed(N + H)
    first = slots_of(g, [((3 * i) % 6, 1) for i in range(N)], N)
    second = [s + 1 for s in first]
    calls = [(*base.tokens(g, N, H), first), (*base.tokens(g, N, H, size=40.0), second)]
    check_store(msa, calls, N, H, N)


# .. 2, 2, 4 and 8 heads
@pytest.mark.parametrize("N,H", [(640, 8), (1024, 8), (1000, 13), (1024, 32)])
def test_runs_of_every_length(msa, N, H):  # noqa: F811
    """Short and long runs from every row, then a token behind each; the rows that are left over store nothing."""
    g = torch.Generator().manual_seed(N * H)
    runs, n = [], 0
    lengths = [1, 2, 8, 9, 3, 17, 5, 40, 7, 128, 4, 6, 64, 1]
    while n < N - 130:
        m = lengths[len(runs) % len(lengths)]
        runs.append(((len(runs) * 5) % (BK - m + 1) // 4, m))
        n += m
    order = torch.randperm(len(runs), generator=g).tolist()
    slots = [page * BK + t + i for page, (t, m) in zip(order, runs) for i in range(m)]
    behind = [page * BK + t + m for page, (t, m) in zip(order, runs) if t + m < BK]
    calls = [(*base.tokens(g, N, H), slots + [-1] * (N - len(slots))),
             (*base.tokens(g, N, H, size=9.0), behind + [-1] * (N - len(behind)))]
    check_store(msa, calls, len(runs), H, N + H)


@pytest.mark.parametrize("B,Hkv,G,k", [(96, 8, 6, 16), (700, 1, 8, 3), (200, 4, 2, 5)])
def test_more_sparse_rows_than_run_at_once(msa, B, Hkv, G, k):  # noqa: F811
    g = torch.Generator().manual_seed(B)
    pool = 40
    cache = base.make_cache(msa, g, pool, Hkv)
    Q = (torch.randn(B, Hkv * G, D, generator=g) * 1.5).bfloat16().cuda()
    pt = torch.stack([torch.randperm(pool, generator=g)[:k] for _ in range(B * Hkv)]).int()
    n = torch.randint(0, k + 1, (B * Hkv,), generator=g).int()
    n[torch.rand(B * Hkv, generator=g) < 0.7] = k
    last = torch.randint(1, BK + 1, (B * Hkv,), generator=g).int()
    ws = torch.zeros(msa.msa_attn_decode_q8_workspace_size(B, Hkv), dtype=torch.uint8, device="cuda")
    args = (msa, Q, cache, pt.cuda(), n.cuda(), last.cuda())
    O, LSE, e = base.run_sparse(*args, ws=ws, zeroed=True)
    assert e == 0
    rows = [[base.places(pt[r].numpy(), np.arange((int(n[r]) - 1) * BK + int(last[r]) if n[r] else 0))
             for r in range(b * Hkv, (b + 1) * Hkv)] for b in range(B)]
    base.check_rows(Q, base.values(cache), rows, (O, LSE))
    again = base.run_sparse(*args, ws=ws, zeroed=True)
    assert np.array_equal(O, again[0]) and np.array_equal(LSE, again[1])


def test_page_copies_beside_other_calls(msa):  # noqa: F811
    """A copy writes its pages anew in every round, on a stream of its own beside decode attention on another one."""
    g = torch.Generator(device="cuda").manual_seed(3)
    P, H, lengths = 60, 4, [3000, 2000, 700]
    pool = torch.randn(2 * P, H, BK, D, generator=g, device="cuda").bfloat16()
    src = torch.randperm(P, generator=g, device="cuda").int()
    dst = torch.arange(P, 2 * P, dtype=torch.int32, device="cuda")
    want = pool[src.long()].clone()
    Q, cache, pt = base.dense_case(msa, lengths, H, 6, 5)
    ptc, L = pt.cuda(), base.dev(lengths, torch.int32)
    O, LSE = torch.zeros(3, H * 6, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, H * 6, device="cuda")
    ws = torch.zeros(msa.msa_attn_decode_q8_workspace_size(3, H), dtype=torch.uint8, device="cuda")
    alone = base.run_dense(msa, Q, cache, pt, lengths)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        pool[P:] = 7
        O.zero_()
        torch.cuda.synchronize()
        msa.msa_dense_attn_decode_q8(Q, cache, ptc, L, O, LSE, ws, stream=b, scratch_zeroed=True)
        msa.msa_copy_pages([pool], src, dst, stream=a)
        torch.cuda.synchronize()
        assert torch.equal(pool[P:], want)
        assert np.array_equal(base.host(O), alone[0])
