"""Requests that share pages on the GPU: forks, their release, compaction and page copies, against serial definitions, and a
run of them over a cache."""
import numpy as np
import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu
BK = 128


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def i32(a):
    return torch.as_tensor(np.asarray(a)).to(device="cuda", dtype=torch.int32)


def num(t):
    return t.cpu().numpy().astype(np.int64)


def requests(seed, lengths, max_pages, extra, shared=0.4):
    """(lengths, table, stack, its height, counts): some requests share the full pages of the one before."""
    rng = np.random.default_rng(seed)
    tables, nxt = [], 0
    for b, L in enumerate(lengths):
        n = -(-L // BK)
        common = min(L, lengths[b - 1]) // BK if b and rng.random() < shared else 0
        tables.append((tables[-1][:common] if common else []) + list(range(nxt, nxt + n - common)))
        nxt += n - common
    P = nxt + extra
    ids = rng.permutation(P)
    pt = np.full((len(lengths), max_pages), -1, np.int64)
    shares = np.zeros(P, np.int64)
    for b, row in enumerate(tables):
        pt[b, :len(row)] = ids[row]
        for j in row:
            shares[ids[j]] += 1
    free = np.full(P, -1, np.int64)
    free[:extra] = ids[nxt:]
    return np.array(lengths, np.int64), pt, free, extra, np.maximum(shares - 1, 0)


def run_fork(msa, src, dst, L, pt, free, count, shares, in_place):
    t = dict(L=i32(L), pt=i32(pt), free=i32(free), count=i32([count]), shares=i32(shares), e=i32([0]))
    o = dict(L=t["L"], pt=t["pt"], count=t["count"], shares=t["shares"]) if in_place else dict(
        L=i32(np.full(len(L), -77)), pt=i32(pt), count=i32([-77]), shares=i32(np.full(len(shares), -77)))
    c = i32(np.full(len(src), -77)), i32(np.full(len(src), -77))
    msa.msa_fork_requests(i32(src), i32(dst), t["L"], t["pt"], t["free"], t["count"], t["shares"], o["L"], o["pt"], o["count"],
                          o["shares"], *c, dev_err=t["e"])
    return dict(seq_len=num(o["L"]), seq_pt=num(o["pt"]), shares=num(o["shares"]), count=int(o["count"]), copy_src=num(c[0]),
                copy_dst=num(c[1]), err=int(t["e"]), free=num(t["free"]))


def check_fork(msa, src, dst, L, pt, free, count, shares):
    want = ref.fork(src, dst, L, pt, free, count, shares)
    for in_place in (False, True):
        got = run_fork(msa, src, dst, L, pt, free, count, shares, in_place)
        for k, v in want.items():
            assert np.array_equal(got[k], v), k
        assert np.array_equal(got["free"], free)
    return want


@pytest.mark.parametrize("seed", range(6))
def test_fork(msa, seed):
    rng = np.random.default_rng(seed)
    B = [4, 9, 33, 200, 700, 4096][seed]
    lengths = [0 if rng.random() < 0.5 else int(rng.integers(1, 3000 if B < 1000 else 600)) for _ in range(B)]
    lengths[0], lengths[-1] = 256, 0
    state = requests(seed, lengths, 26, B)
    live, empty = np.flatnonzero(state[0] > 0), np.flatnonzero(state[0] == 0)
    F = len(empty)
    dst = rng.permutation(empty)
    src = rng.choice(live, F)
    src[rng.random(F) < 0.2] = -1                         # padding
    assert check_fork(msa, src, dst, *state)["err"] == 0


def test_fork_refusals(msa):
    L, pt, free, count, shares = requests(1, [300, 0, 128, 0, 0, 700, 0, 0, 0, 0], 6, 4)
    pt[5, 1] = len(shares) + 3                            # handed on, not counted
    L2 = L.copy()
    L2[2] = 6 * BK + 1
    src = [0, 0, 10, 0, 0, 2, 5, 5, -1, 5, 5, 0, 1, 0]
    dst = [1, 1, 3, 10, 5, 3, 4, 6, 7, 7, 8, 9, 9, 3]
    want = check_fork(msa, src, dst, L2, pt, free, count, shares)
    assert want["err"] == msa.MSA_DEVERR_BAD_ROW | msa.MSA_DEVERR_BAD_LEN | msa.MSA_DEVERR_BAD_PAGE | msa.MSA_DEVERR_NO_PAGES
    check_fork(msa, [0], [1], L, pt, free, 99, shares)    # a stack's height outside it
    check_fork(msa, [0], [1], L, pt, free, -2, shares)
    check_fork(msa, [], [], L, pt, free, count, shares)


def run_release(msa, L, done, pt, free, count, shares, in_place):
    t = dict(L=i32(L), free=i32(free), count=i32([count]), shares=i32(shares), e=i32([0]))
    o = dict(L=t["L"], count=t["count"], shares=t["shares"]) if in_place else dict(
        L=i32(np.full(len(L), -77)), count=i32([-77]), shares=i32(np.full(len(shares), -77)))
    msa.msa_release_shared_pages(t["L"], i32(done), i32(pt), t["free"], t["count"], t["shares"], o["L"], o["count"], o["shares"],
                                 dev_err=t["e"])
    return dict(seq_len=num(o["L"]), free=num(t["free"]), count=int(o["count"]), shares=num(o["shares"]), err=int(t["e"]))


def check_release(msa, *state):
    want = ref.release_shared(*state)
    for in_place in (False, True):
        got = run_release(msa, *state, in_place)
        for k, v in want.items():
            assert np.array_equal(got[k], v), k
    return want


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("shared", [0.0, 0.8])
def test_release(msa, seed, shared):
    rng = np.random.default_rng(seed)
    B = [1, 5, 40, 300, 900, 4096][seed]
    lengths = [int(rng.integers(0, 5000 if B < 1000 else 400)) for _ in range(B)]
    L, pt, free, count, shares = requests(seed, lengths, 40, 7, shared)
    done = (rng.random(B) < 0.6).astype(np.int64)
    assert check_release(msa, L, done, pt, free, count, shares)["err"] == 0
    want = check_release(msa, L, np.ones(B, np.int64), pt, free, count, shares)
    assert want["err"] == 0 and want["count"] == len(shares) and not want["shares"].any()


def test_release_refusals(msa):
    L, pt, free, count, shares = requests(3, [300, 200, 128, 700], 6, 2, 1.0)
    pt2 = pt.copy()
    pt2[3, 3], pt2[1, 1] = -4, pt[0, 2]                   # out of the pool; a page that its count says is not shared
    L2 = L.copy()
    L2[2] = -5
    want = check_release(msa, L2, np.ones(4, np.int64), pt2, free, count, shares)
    assert want["err"] == msa.MSA_DEVERR_BAD_PAGE | msa.MSA_DEVERR_BAD_LEN
    assert check_release(msa, L, np.ones(4, np.int64), pt, free[:4], count, shares)["err"] == msa.MSA_DEVERR_NO_PAGES
    check_release(msa, L, np.ones(4, np.int64), pt, free, len(free) + 5, shares)


def run_compact(msa, L, pt, shares, cap, in_place):
    t = dict(L=i32(L), pt=i32(pt), shares=i32(shares), e=i32([0]))
    pt_out, s_out = (t["pt"], t["shares"]) if in_place else (i32(np.full(pt.shape, -77)), i32(np.full(len(shares), -77)))
    free, count = i32(np.full(cap, -77)), i32([-77])
    mv = i32(np.full(len(shares), -77)), i32(np.full(len(shares), -77))
    msa.msa_compact_pages(t["L"], t["pt"], t["shares"], pt_out, s_out, free, count, *mv, dev_err=t["e"])
    return dict(pt=num(pt_out), shares=num(s_out), free=num(free), count=int(count), move_src=num(mv[0]), move_dst=num(mv[1]), err=int(t["e"]))


def check_compact(msa, L, pt, shares, cap):
    want = ref.compact(L, pt, shares, cap)
    for in_place in (False, True):
        got = run_compact(msa, L, pt, shares, cap, in_place)
        for k in ("shares", "free", "count", "move_src", "move_dst", "err"):
            assert np.array_equal(got[k], want[k]), k
        table = pt.copy() if in_place else np.full(pt.shape, -77)
        for at, page in want["entries"].items():
            table[at] = page
        assert np.array_equal(got["pt"], table)
    return want


@pytest.mark.parametrize("seed,B,extra", [(0, 1, 0), (1, 1, 5), (2, 6, 50), (3, 40, 1), (4, 40, 3000), (5, 500, 0), (6, 4096, 777), (7, 3, 70000)])
def test_compact(msa, seed, B, extra):
    rng = np.random.default_rng(seed)
    lengths = [int(rng.integers(0, 4000 if B < 1000 else 300)) for _ in range(B)]
    L, pt, free, count, shares = requests(seed, lengths, 32, max(extra, 1 if sum(lengths) == 0 else 0), 0.5)
    want = check_compact(msa, L, pt, shares, len(shares) + seed)
    assert want["err"] == 0


def test_compact_refusals_and_nothing_to_do(msa):
    L, pt, free, count, shares = requests(8, [300, 200, 128, 700], 6, 30)
    pt[0, 1], pt[3, 5] = -4, len(shares)
    L[1] = 6 * BK + 1
    assert check_compact(msa, L, pt, shares, len(shares))["err"] == msa.MSA_DEVERR_BAD_LEN | msa.MSA_DEVERR_BAD_PAGE
    check_compact(msa, np.zeros(4, np.int64), pt, shares, len(shares))
    pt = np.arange(24).reshape(4, 6)                      # the whole pool in use
    check_compact(msa, np.full(4, 6 * BK), pt, np.zeros(24, np.int64), 24)


# ---------------------------------------------------------------------------
# copies
# ---------------------------------------------------------------------------

def test_copy_pages(msa):
    g = torch.Generator().manual_seed(0)
    P = 50
    wide = torch.randn(P, 3, 2, BK, 128, generator=g).bfloat16().cuda()
    pools = [wide[:, 0], wide[:, 2],                       # pages contiguous, the pools not
             torch.randint(0, 255, (P, 5), dtype=torch.uint8, generator=g).cuda(), torch.randn(P, 7, 33, generator=g).cuda(),
             torch.randint(0, 255, (P, 16 * 1024 + 16), dtype=torch.uint8, generator=g).cuda(), torch.randn(P, generator=g).cuda(),
             torch.randn(P, 2, 4096, generator=g).half().cuda()]
    want = [p.clone() for p in pools]
    untouched = wide[:, 1].clone()
    perm = torch.randperm(P, generator=g)
    src, dst = perm[:20].clone(), perm[20:40].clone()
    src[5], dst[5] = src[4], dst[5]                        # a source named twice
    for w in want:
        w[dst.cuda()] = w[src.cuda()]
    s = torch.full((90,), -1, dtype=torch.int32)
    d = torch.full((90,), -1, dtype=torch.int32)
    at = torch.randperm(90, generator=g)[:20]
    s[at], d[at] = src.int(), dst.int()
    free = [i for i in range(90) if i not in at.tolist()]
    s[free[0]] = 3                                         # no target: left out
    d[free[1]] = int(perm[45])                             # no source: left out
    e = i32([0])
    msa.msa_copy_pages(pools, s.cuda(), d.cuda(), dev_err=e)
    assert int(e) == 0
    for p, w in zip(pools, want):
        assert torch.equal(p, w)
    assert torch.equal(wide[:, 1], untouched)
    msa.msa_copy_pages(tuple(pools), i32([P, 1, -3]), i32([2, P + 9, 4]), dev_err=e)
    assert int(e) == msa.MSA_DEVERR_BAD_PAGE
    for p, w in zip(pools, want):
        assert torch.equal(p, w)
    msa.msa_copy_pages([], i32([0]), i32([1]))
    msa.msa_copy_pages(pools, i32([]), i32([]))


def test_many_copies(msa):
    g = torch.Generator().manual_seed(1)
    P = 3000
    pool = torch.randint(0, 1 << 30, (P, 1000), dtype=torch.int32, generator=g).cuda()
    perm = torch.randperm(P, generator=g).cuda().int()
    want = pool.clone()
    want[perm[1500:].long()] = want[perm[:1500].long()]
    msa.msa_copy_pages([pool], perm[:1500], perm[1500:])
    assert torch.equal(pool, want)


# ---------------------------------------------------------------------------
# a run of them over an 8-bit cache
# ---------------------------------------------------------------------------

def test_a_run(msa):
    """Prompts stored, continued by several samples that share them, samples that end, a compaction: attention over the cache
    reads the same tokens as a cache that every request has to itself.  Captured and replayed, too."""
    g = torch.Generator().manual_seed(2)
    B, P, Hkv, G, mp = 8, 40, 2, 3, 8
    text = [[] for _ in range(B)]                          # (K, V) tokens of every request
    cache = msa.q8_cache(P, Hkv, "cuda")
    L, done, new = i32([0] * B), i32([0] * B), i32([0] * B)
    pt, free, count, shares = i32(np.full((B, mp), -1)), i32(np.arange(P)), i32([P]), i32([0] * P)
    plan, err = msa.plan_buffers(B, 600, "cuda"), i32([0])
    plan["seq_len_out"], plan["free_count_out"] = L, count
    F = 4
    src, dst, cs, cd = i32([-1] * F), i32([-1] * F), i32([-1] * F), i32([-1] * F)
    K, V = (torch.zeros(600, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mv, stack = [i32([-1] * P) for _ in range(2)], i32([-1] * P)
    pools = [cache.K_codes, cache.K_scales, cache.V_codes, cache.V_scales]

    def step():
        msa.msa_release_shared_pages(L, done, pt, free, count, shares, L, count, shares, dev_err=err)
        msa.msa_fork_requests(src, dst, L, pt, free, count, shares, L, pt, count, shares, cs, cd, dev_err=err)
        msa.msa_copy_pages(pools, cs, cd, dev_err=err)
        msa.msa_plan_step(L, new, pt, free, count, L, count, plan["cu"], plan["tok_slot"], plan["tok_pos"], plan["tok_seq"],
                          num_pages=P, dev_err=err)
        msa.msa_cache_append_q8(K, V, plan["tok_slot"], cache, dev_err=err)

    def compact():
        msa.msa_compact_pages(L, pt, shares, pt, shares, stack, count, *mv, dev_err=err)
        msa.msa_copy_pages(pools, *mv, dev_err=err)
        free.copy_(stack)

    side = torch.cuda.Stream()                             # (a capture wants modules loaded)
    with torch.cuda.stream(side):
        step()
        compact()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for graph, f in zip(graphs, (step, compact)):
        with torch.cuda.graph(graph):
            f()

    def play(ended, forks, fresh, how):
        done.copy_(i32([int(b in ended) for b in range(B)]))
        s, d = [f[0] for f in forks] + [-1] * (F - len(forks)), [f[1] for f in forks] + [-1] * (F - len(forks))
        src.copy_(i32(s))
        dst.copy_(i32(d))
        for b in ended:
            text[b] = []
        for a, b in forks:
            text[b] = list(text[a])
        counts = [fresh.get(b, 0) for b in range(B)]
        new.copy_(i32(counts))
        at = 0
        for b, n in enumerate(counts):
            for _ in range(n):
                k, v = (torch.randn(Hkv, 128, generator=g).bfloat16() for _ in range(2))
                K[at], V[at] = k.cuda(), v.cuda()
                text[b].append((k, v))
                at += 1
        how()
        torch.cuda.synchronize()
        assert int(err) == 0
        lengths = num(L).tolist()
        assert lengths == [len(x) for x in text]
        held = {p for b in range(B) for p in num(pt)[b, :-(-lengths[b] // BK)].tolist()}
        assert int(count) == P - len(held) and not held & set(num(free)[:int(count)].tolist())
        # every request's tokens are where its table says, in 8 bits (half a step, twice where a block was rounded again)
        kv = [ref.decode(c.cpu().numpy(), s.cpu().numpy()[..., None, None]) for c, s in ((cache.K_codes, cache.K_scales), (cache.V_codes, cache.V_scales))]
        for b, x in enumerate(text):
            for t, kvs in enumerate(x):
                p = num(pt)[b, t // BK]
                for have, want in zip(kv, kvs):
                    w = want.double().numpy()
                    assert np.all(np.abs(have[p, :, t % BK] - w) <= np.abs(w) * 2.0 ** -3 + 2.0 ** -9)
        Q = torch.randn(B, Hkv * G, 128, generator=g).bfloat16().cuda()
        O, LSE = torch.empty_like(Q), torch.empty(B, Hkv * G, device="cuda")
        msa.msa_dense_attn_decode_q8(Q, cache, pt, L, O, LSE, torch.zeros(msa.msa_attn_decode_q8_workspace_size(B, Hkv), dtype=torch.uint8,
                                                                            device="cuda"), dev_err=err)
        o, lse, q, table = O.double().cpu().numpy(), LSE.double().cpu().numpy(), Q.double().cpu().numpy(), num(pt)
        for b, n in enumerate(lengths):
            t = np.arange(n)
            for h in range(Hkv):
                hs = slice(h * G, (h + 1) * G)
                k, v = (x[table[b, t // BK], h, t % BK] for x in kv)
                ref.check(o[b, hs], lse[b, hs], ref.attend(q[b, hs], k, v, 128 ** -0.5), ref.HALF["fp16"])

    for how_step, how_compact in ((step, compact), (graphs[0].replay, graphs[1].replay)):
        play(set(), [], {0: 300, 1: 128}, how_step)
        play(set(), [(0, 2), (0, 3), (1, 4)], {0: 1, 2: 1, 3: 1, 4: 1}, how_step)
        play({0}, [(2, 5)], {2: 1, 3: 100, 4: 1, 5: 1}, how_step)
        play(set(), [], {}, how_compact)
        play({2, 3}, [(5, 0), (4, 2)], {0: 1, 1: 1, 2: 130, 4: 1, 5: 1}, how_step)
        play(set(), [], {}, how_compact)
        play({0, 1, 2, 4, 5}, [], {}, how_step)
        assert int(count) == P and not num(shares).any()
