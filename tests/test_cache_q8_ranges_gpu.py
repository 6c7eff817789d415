"""Decode attention over 8-bit pages whose blocks of V differ by up to 2^80: every channel is as exact as the tokens that fill
it, whatever the other channels and blocks hold.

Each page fills a set of channels of its own, so that a channel's output is that of one or two pages.  A token's weight is
p / l, p = exp(z - max z).  It enters the products as 2^8 p in fp16, with up to 2^-8 more for a block of smaller values, so it
is off by half a step, 2^-11 of it, or by half a subnormal step: 2^-25 of the largest token's weight.  Scores, exponentials
and sums in fp32 as in cache_ref.check, and the output's own rounding to bf16."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import test_cache_q8_gpu as base
from test_cache_q8_gpu import msa  # noqa: F401

pytestmark = pytest.mark.gpu
BK, D = 128, 128


def own_channels(cache, lists, order, g):
    """V blocks of the j-th page of every list fill channels j, j + n, ..; their scales fall, rise, or go either way."""
    for pages in lists:
        n = len(pages)
        span = np.linspace(167, 87, n).round().astype(int) if n > 1 else np.array([127])
        at = {"falling": span, "rising": span[::-1], "mixed": span[torch.randperm(n, generator=g).numpy()],
              "first": np.array([167] + [127] * (n - 1)), "near": 127 + np.arange(n) % 10}[order]
        for j, page in enumerate(pages):
            keep = torch.zeros(D, dtype=torch.bool)
            keep[j % min(n, D)::min(n, D)] = True
            cache.V_codes[page][..., ~keep] = 0
            cache.V_scales[page] = int(at[j])


def check_channels(Q, kv, rows, got):
    O, LSE = got
    q, scale = base.host(Q), 1 / np.sqrt(D)
    for b, heads in enumerate(rows):
        G = q.shape[1] // len(heads)
        for g, (pages, at) in enumerate(heads):
            if len(pages) == 0:
                assert np.all(O[b, g * G:(g + 1) * G] == 0) and np.all(np.isneginf(LSE[b, g * G:(g + 1) * G]))
                continue
            K, V, x = kv[0][pages, g, at], kv[1][pages, g, at], q[b, g * G:(g + 1) * G]
            z = x @ K.T * scale
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            l = p.sum(1, keepdims=True)
            o, lse = p @ V / l, (m + np.log(l))[:, 0]
            near = (np.abs(x) @ np.abs(K).T).max(1, keepdims=True) * scale * 2.0 ** -19 + 2.0 ** -17
            tol = (2.0 ** -8 * np.abs(o) + (2.0 ** -11 + near) * (p @ np.abs(V) / l)) * (1 + 2.0 ** -7) + 2.0 ** -25 * np.abs(V).sum(0) / l
            at_head = slice(g * G, (g + 1) * G)
            bad = ~(np.abs(O[b, at_head] - o) <= tol)
            assert not bad.any(), (b, g, np.argwhere(bad)[:4], O[b, at_head][bad][:4], o[bad][:4], tol[bad][:4])
            assert np.all(np.abs(LSE[b, at_head] - lse) <= near[:, 0] + 2.0 ** -22 * np.abs(lse))


@pytest.mark.parametrize("order", ["first", "falling", "rising", "mixed", "near"])
@pytest.mark.parametrize("q", [0.0, 1.5])
@pytest.mark.parametrize("B,Hkv,G,k", [(1, 1, 8, 16), (3, 2, 6, 5), (40, 4, 3, 16), (90, 8, 1, 4)])
def test_sparse(msa, order, q, B, Hkv, G, k):  # noqa: F811
    g = torch.Generator().manual_seed(B + k)
    pool = 2 * k
    cache = base.make_cache(msa, g, pool, Hkv)
    own_channels(cache, [list(range(k)), list(range(k, 2 * k))], order, g)
    Q = (torch.randn(B, Hkv * G, D, generator=g) * q).bfloat16().cuda()
    pt = torch.stack([torch.arange(k) + k * (r % 2) for r in range(B * Hkv)]).int()
    n = torch.full((B * Hkv,), k, dtype=torch.int32)
    last = torch.randint(1, BK + 1, (B * Hkv,), generator=g).int()
    if B > 1:
        n[-1], n[-2] = 0, 1
    O, LSE, e = base.run_sparse(msa, Q, cache, pt.cuda(), n.cuda(), last.cuda())
    assert e == 0
    rows = [[base.places(pt[r].numpy(), np.arange(max(0, (int(n[r]) - 1) * BK + int(last[r])) if n[r] else 0))
             for r in range(b * Hkv, (b + 1) * Hkv)] for b in range(B)]
    check_channels(Q, base.values(cache), rows, (O, LSE))


@pytest.mark.parametrize("order", ["first", "falling", "rising", "mixed", "near"])
@pytest.mark.parametrize("lengths,Hkv,G,window,sinks", [
    ([1500], 1, 4, 0, 0), ([20000, 700], 2, 6, 0, 0), ([900, 0, 1, 1300] * 30, 4, 2, 0, 0), ([3000, 140], 2, 8, 900, 130),
    ([9000] * 3, 4, 6, 8500, 4), ([800] * 100, 4, 1, 600, 20)])
def test_dense_and_windows(msa, order, lengths, Hkv, G, window, sinks):  # noqa: F811
    Q, cache, pt = base.dense_case(msa, lengths, Hkv, G, len(lengths) + G)
    g = torch.Generator().manual_seed(7)
    own_channels(cache, [pt[b, :-(-L // BK)].tolist() for b, L in enumerate(lengths)], order, g)
    for q in (0.0, 1.0):
        x = Q * q
        O, LSE, e = base.run_dense(msa, x, cache, pt, lengths, window, sinks)
        assert e == 0
        rows = [[base.places(pt[b].numpy(), ref.seen(L - 1, window, sinks))] * Hkv for b, L in enumerate(lengths)]
        check_channels(x, base.values(cache), rows, (O, LSE))


def test_large_values_of_one_token(msa):  # noqa: F811
    """One token of 448 * 2^40 in one channel, all others of ordinary size: the other channels are the mean of theirs."""
    lengths = [640] * 120
    Q, cache, pt = base.dense_case(msa, lengths, 4, 2, 9)
    Q.zero_()
    cache.V_scales.fill_(120)
    for b in range(len(lengths)):
        page = pt[b, b % 5].item()
        cache.V_codes[page] = 0
        cache.V_codes[page, :, 17, 3] = 0x7E
        cache.V_scales[page] = 167
    O, LSE, e = base.run_dense(msa, Q, cache, pt, lengths)
    assert e == 0
    check_channels(Q, base.values(cache), [[base.places(pt[b].numpy(), np.arange(L))] * 4 for b, L in enumerate(lengths)], (O, LSE))


@pytest.mark.parametrize("order", ["first", "mixed"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
def test_anything_in_slots_that_are_not_seen(msa, order, window, sinks):  # noqa: F811
    """Blocks far apart, NaN codes in every slot that no query sees: nothing changes."""
    lengths = [700, 1290, 40] * 40
    Q, cache, pt = base.dense_case(msa, lengths, 2, 6, 4)
    g = torch.Generator().manual_seed(8)
    own_channels(cache, [pt[b, :-(-L // BK)].tolist() for b, L in enumerate(lengths)], order, g)
    want = base.run_dense(msa, Q, cache, pt, lengths, window, sinks)
    for b, L in enumerate(lengths):
        hidden = np.setdiff1d(np.arange(-(-L // BK) * BK), ref.seen(L - 1, window, sinks))
        page, row = (torch.as_tensor(x, device="cuda").long() for x in base.places(pt[b].numpy(), hidden))
        cache.K_codes[page, :, row] = 0x7F
        cache.V_codes[page, :, row] = 0xFF
    got = base.run_dense(msa, Q, cache, pt, lengths, window, sinks)
    assert got[2] == 0 and np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
