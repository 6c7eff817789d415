"""The 8-bit paged cache on the GPU: store, expansion, sparse and dense decode attention, and a step of them, against
64-bit definitions."""
import math

import numpy as np
import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu
BK, D = 128, 128


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def dev(a, dtype=None):
    return torch.as_tensor(np.asarray(a)).to(device="cuda", dtype=dtype)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def make_cache(msa, g, pages, H, spread=0.5, strided=False):
    """A cache of random codes (no NaN) and scale bytes, as pool views with gaps if `strided`."""
    def pool(*shape):
        if strided:
            return torch.zeros(pages, H + 1, *[s if i else s for i, s in enumerate(shape)], dtype=torch.uint8, device="cuda")[:, 1:]
        return torch.zeros(pages, H, *shape, dtype=torch.uint8, device="cuda")
    c = msa.Q8Cache(pool(BK, D), pool(), pool(BK, D), pool())
    for codes, scales, mid in ((c.K_codes, c.K_scales, 121), (c.V_codes, c.V_scales, 120)):
        x = torch.randn(pages, H, BK, D, generator=g) * 60
        codes.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        scales.copy_((mid + torch.randn(pages, H, generator=g) * spread * 2).round().clamp(87, 167).to(torch.uint8))
    return c


def values(cache):
    """K and V of the whole cache in 64 bits [P, H, BK, D]."""
    return [ref.decode(c.cpu().numpy(), s.cpu().numpy()[..., None, None])
            for c, s in ((cache.K_codes, cache.K_scales), (cache.V_codes, cache.V_scales))]


# ---------------------------------------------------------------------------
# store and expansion
# ---------------------------------------------------------------------------

def check_store(msa, calls, pages, H, strided=False, seed=0):
    """Every call's (K, V, slots) into the cache, against the serial definition, byte for byte; then all pages expanded."""
    g = torch.Generator().manual_seed(seed)
    cache = make_cache(msa, g, pages, H, strided=strided)
    want = [[c.cpu().numpy().copy(), s.cpu().numpy().copy()] for c, s in ((cache.K_codes, cache.K_scales), (cache.V_codes, cache.V_scales))]
    for K, V, slots in calls:
        e = err_word()
        msa.msa_cache_append_q8(K.cuda(), V.cuda(), dev(slots, torch.int64), cache, dev_err=e)
        bad = any(s >= pages * BK for s in slots)
        assert int(e.item()) == (msa.MSA_DEVERR_BAD_PAGE if bad else 0)
        for (codes, scales), x in zip(want, (K, V)):
            ref.store(codes, scales, x.double().numpy(), np.asarray(slots))
        for (codes, scales), c, s in zip(want, (cache.K_codes, cache.V_codes), (cache.K_scales, cache.V_scales)):
            assert np.array_equal(s.cpu().numpy(), scales)
            assert np.array_equal(c.cpu().numpy(), codes)
    ids = torch.randperm(pages, generator=g).int()
    out = [torch.full((pages, H, BK, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    msa.msa_cache_expand_q8(cache, ids.cuda(), *out)
    for (codes, scales), o in zip(want, out):
        v = ref.decode(codes, scales[..., None, None])[ids.numpy()]
        assert np.array_equal(host(o), v, equal_nan=True)


def tokens(g, n, H, size=1.0):
    return ((torch.randn(n, H, D, generator=g) * size).bfloat16(), (torch.randn(n, H, D, generator=g) * size * 0.3).bfloat16())


@pytest.mark.parametrize("lengths", [[1], [8], [9], [31, 33], [127], [128], [129], [1, 2, 3, 7, 8, 9, 40], [300, 1, 513]])
@pytest.mark.parametrize("start", [0, 1, 77, 127])
def test_runs(msa, lengths, start):
    g = torch.Generator().manual_seed(sum(lengths) + start)
    slots, page = [], 0
    order = torch.randperm(32, generator=g).tolist()
    for n in lengths:
        t = start
        for _ in range(n):
            slots.append(order[page] * BK + t)
            t += 1
            if t == BK:
                t, page = 0, page + 1
        page += 1
    check_store(msa, [(*tokens(g, len(slots), 3), slots)], 32, 3)


def test_token_by_token(msa):
    """A block that fills one token at a time, each larger than the ones before for a while: its scale grows, the rows before
    are rounded again; then the page starts anew."""
    g = torch.Generator().manual_seed(5)
    calls = []
    for t in list(range(0, 128, 3)) + [0, 1]:
        K, V = tokens(g, 2, 2, size=2.0 ** (t / 4 - 10))
        calls.append((K, V, [5 * BK + t, 1 * BK + t]))
    check_store(msa, calls, 6, 2)


def test_many_sequences_of_one_token_and_a_chunk(msa):
    g = torch.Generator().manual_seed(6)
    slots = [p * BK + (p * 37) % BK for p in range(100)] + [100 * BK + i for i in range(1500)]
    check_store(msa, [(*tokens(g, 1600, 2), slots)], 120, 2)


def test_left_out_rows_and_bad_slots(msa):
    g = torch.Generator().manual_seed(7)
    slots = [-1, 3 * BK + 5, 3 * BK + 6, -1, -7, 9 * BK, 2 * BK + 127, 4 * BK, 8 * BK - 1, 1 << 40]
    check_store(msa, [(*tokens(g, len(slots), 2), slots)], 8, 2)


def test_special_values(msa):
    """Zeros, infinities, NaN, the smallest and largest magnitudes; blocks of only those."""
    g = torch.Generator().manual_seed(8)
    K, V = tokens(g, 12, 2)
    for i, v in enumerate((0.0, math.inf, -math.inf, math.nan, 3.3e38, -3.3e38, 1e-38, 9e-41, 448.0, 464.0, 2.0 ** -49)):
        K[i] = v
        V[i, 0, i] = v
    slots = [i * BK + (5 * i) % 7 for i in range(12)]
    check_store(msa, [(K, V, slots)], 12, 2)


def test_strided_inputs_and_pools(msa):
    g = torch.Generator().manual_seed(9)
    K, V = tokens(g, 40, 6)
    check_store(msa, [(K[::2, 1:5:2], V[::2, 1:5:2], [2 * BK + i for i in range(20)])], 4, 2, strided=True)


def test_expand_leaves_bad_pages(msa):
    g = torch.Generator().manual_seed(10)
    cache = make_cache(msa, g, 4, 2)
    out = [torch.full((3, 2, BK, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    e = err_word()
    msa.msa_cache_expand_q8(cache, dev([4, 1, -1], torch.int32), *out, dev_err=e)
    assert int(e.item()) == msa.MSA_DEVERR_BAD_PAGE
    for o, v in zip(out, values(cache)):
        assert bool((o[0] == 7).all()) and bool((o[2] == 7).all())
        assert np.array_equal(host(o[1]), v[1])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def run_sparse(msa, Q, cache, pt, n, last, scale=0.0, zeroed=False, ws=None):
    B, Hq, _ = Q.shape
    O = torch.full((B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((B, Hq), 7.0, device="cuda")
    if ws is None:
        ws = torch.zeros(msa.msa_attn_decode_q8_workspace_size(B, pt.shape[0] // B), dtype=torch.uint8, device="cuda")
    e = err_word()
    msa.msa_sparse_attn_decode_q8(Q, cache, pt, n, last, O, LSE, ws, softmax_scale=scale, dev_err=e, scratch_zeroed=zeroed)
    return host(O), LSE.double().cpu().numpy(), int(e.item())


def check_rows(Q, kv, rows, got, scale=1 / math.sqrt(D), half=ref.HALF["fp16"]):
    """rows[b][g]: (pages, rows within them) of the tokens that sequence b's query sees."""
    O, LSE = got
    q = host(Q)
    for b, heads in enumerate(rows):
        G = q.shape[1] // len(heads)
        for g, (pages, at) in enumerate(heads):
            h = slice(g * G, (g + 1) * G)
            ref.check(O[b, h], LSE[b, h], ref.attend(q[b, h], kv[0][pages, g, at], kv[1][pages, g, at], scale), half)


def places(pages, tokens):
    """(page, row) of these tokens of a page list."""
    return np.asarray(pages)[tokens // BK], tokens % BK


@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 3), (8, 6), (4, 8), (3, 5)])
@pytest.mark.parametrize("k", [1, 3, 16, 40, 64])
def test_sparse(msa, Hkv, G, k):
    g = torch.Generator().manual_seed(k * 100 + G)
    B, pool = 3, 70
    cache = make_cache(msa, g, pool, Hkv)
    Q = (torch.randn(B, Hkv * G, D, generator=g) * 1.5).bfloat16().cuda()
    pt = torch.stack([torch.randperm(pool, generator=g)[:k] for _ in range(B * Hkv)]).int()
    n = torch.randint(0, k + 1, (B * Hkv,), generator=g).int()
    last = torch.randint(0, BK + 1, (B * Hkv,), generator=g).int()
    n[0], last[0], n[-1], last[-1] = k, BK, k, 1
    O, LSE, e = run_sparse(msa, Q, cache, pt.cuda(), n.cuda(), last.cuda())
    assert e == 0
    kv, rows = values(cache), []
    for b in range(B):
        rows.append([])
        for h in range(Hkv):
            r = b * Hkv + h
            T = max(0, (int(n[r]) - 1) * BK + int(last[r])) if n[r] else 0
            rows[-1].append(places(pt[r].numpy(), np.arange(T)))
    check_rows(Q, kv, rows, (O, LSE))


def dense_case(msa, lengths, Hkv, G, seed, spread=0.5, max_pages=None):
    g = torch.Generator().manual_seed(seed)
    per = [-(-L // BK) for L in lengths]
    pool = sum(per) + 3
    cache = make_cache(msa, g, pool, Hkv, spread)
    ids = torch.randperm(pool, generator=g).int()
    pt = torch.full((len(lengths), max_pages or max(max(per), 1)), -1, dtype=torch.int32)
    for b, n in enumerate(per):
        pt[b, :n] = ids[sum(per[:b]):sum(per[:b + 1])]
    Q = (torch.randn(len(lengths), Hkv * G, D, generator=g) * 1.5).bfloat16().cuda()
    return Q, cache, pt


def run_dense(msa, Q, cache, pt, lengths, window=0, sinks=0, ws=None, zeroed=False, stream=None):
    B, Hq, _ = Q.shape
    O = torch.full((B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((B, Hq), 7.0, device="cuda")
    if ws is None:
        ws = torch.zeros(msa.msa_attn_decode_q8_workspace_size(B, cache.K_codes.shape[1]), dtype=torch.uint8, device="cuda")
    e = err_word()
    msa.msa_dense_attn_decode_q8(Q, cache, pt.cuda(), dev(lengths, torch.int32), O, LSE, ws, window=window, sinks=sinks, dev_err=e,
                                 scratch_zeroed=zeroed, stream=stream)
    return host(O), LSE.double().cpu().numpy(), int(e.item())


def check_dense(Q, cache, pt, lengths, got, window=0, sinks=0):
    kv, Hkv = values(cache), cache.K_codes.shape[1]
    rows = [[places(pt[b].numpy(), ref.seen(L - 1, window, sinks))] * Hkv for b, L in enumerate(lengths)]
    check_rows(Q, kv, rows, got)


@pytest.mark.parametrize("lengths,Hkv,G", [
    ([1], 1, 1), ([15, 16, 17], 2, 6), ([127, 128, 129, 1], 4, 3), ([0, 2000, 0, 64], 2, 8), ([9000], 1, 4), ([5000, 5001], 8, 6),
    ([33] * 40, 8, 2), (list(range(1, 700, 7)), 2, 5), ([60000], 1, 1), ([20000] * 3 + [1], 4, 6), ([300] * 300, 2, 1)])
def test_dense(msa, lengths, Hkv, G):
    Q, cache, pt = dense_case(msa, lengths, Hkv, G, len(lengths) + G)
    O, LSE, e = run_dense(msa, Q, cache, pt, lengths)
    assert e == 0
    check_dense(Q, cache, pt, lengths, (O, LSE))
    again = run_dense(msa, Q, cache, pt, lengths)
    assert np.array_equal(O, again[0]) and np.array_equal(LSE, again[1])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (128, 128), (129, 130), (1000, 300), (5000, 0), ((1 << 31) - 1, 3),
                                          (2000, 1 << 30)])
@pytest.mark.parametrize("lengths,Hkv,G", [([1, 2, 16, 130, 0, 700, 3000], 2, 6), ([9000], 1, 8), ([500] * 100, 4, 3)])
def test_window(msa, window, sinks, lengths, Hkv, G):
    Q, cache, pt = dense_case(msa, lengths, Hkv, G, window % 1000 + sinks % 1000)
    O, LSE, e = run_dense(msa, Q, cache, pt, lengths, window, sinks)
    assert e == 0
    check_dense(Q, cache, pt, lengths, (O, LSE), window, sinks)


def test_blocks_of_very_different_sizes(msa):
    """Scales from 2^-40 to 2^40: neither large nor small blocks' values drown or overflow the others' weights."""
    lengths = [700, 128, 1000]
    Q, cache, pt = dense_case(msa, lengths, 2, 4, 77)
    cache.V_scales.copy_(torch.randint(87, 168, cache.V_scales.shape, generator=torch.Generator().manual_seed(1)))
    got = run_dense(msa, Q, cache, pt, lengths)
    check_dense(Q, cache, pt, lengths, got[:2])
    # all weight on a block of small values beside one of large values
    cache.V_scales.fill_(167)
    cache.V_scales[pt[0, 2].item()] = 87
    cache.K_codes.zero_()
    cache.K_scales.fill_(127)
    Q.fill_(1.0)
    p = pt[0, 2].item()
    cache.K_codes[p, :, 5] = 0x50                       # 8.0 in every channel of one token: score 1024 / sqrt(128) against 0
    got = run_dense(msa, Q[:1], cache, pt[:1], lengths[:1])
    check_dense(Q[:1], cache, pt[:1], lengths[:1], got[:2])
    assert np.isfinite(got[0]).all()


@pytest.mark.parametrize("size", [1e4, 1e9, 1e18])
def test_scores_of_any_size(msa, size):
    """Equal keys have equal weights, however large the scores."""
    lengths = [300]
    Q, cache, pt = dense_case(msa, lengths, 1, 2, 3)
    cache.K_codes.fill_(0x38)                           # 1.0
    cache.K_scales.fill_(127)
    Q.fill_(size)
    O, LSE, e = run_dense(msa, Q, cache, pt, lengths)
    v = values(cache)[1][pt[0].numpy(), 0].reshape(-1, D)[:300]
    assert np.all(np.abs(O[0] - v.mean(0)) <= np.abs(v.mean(0)) * 2.0 ** -8 + np.abs(v).mean(0) * 2.0 ** -10)
    z = float(torch.tensor(size).bfloat16()) * math.sqrt(128.0)
    assert np.all(np.abs(LSE - (z + math.log(300))) <= z * 2.0 ** -20 + 1e-4)


def test_anything_behind_the_last_token(msa):
    """NaN codes and NaN scales' neighbours in slots that no query sees change nothing."""
    lengths, window, sinks = [130, 513, 40], 100, 3
    for w, s in ((0, 0), (window, sinks)):
        Q, cache, pt = dense_case(msa, lengths, 2, 6, 4)
        want = run_dense(msa, Q, cache, pt, lengths, w, s)
        for b, L in enumerate(lengths):
            see = set(ref.seen(L - 1, w, s).tolist())
            for t in range(-(-L // BK) * BK):
                if t not in see:
                    cache.K_codes[pt[b, t // BK].item(), :, t % BK] = 0x7F
                    cache.V_codes[pt[b, t // BK].item(), :, t % BK] = 0xFF
        got = run_dense(msa, Q, cache, pt, lengths, w, s)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_bad_lengths_and_pages(msa):
    lengths = [200, 400, 300]
    Q, cache, pt = dense_case(msa, lengths, 2, 3, 5)
    pt[1, 1], pt[2, 0] = cache.K_codes.shape[0], -5
    O, LSE, e = run_dense(msa, Q, cache, pt, [-1, 400, 300])
    assert e == msa.MSA_DEVERR_BAD_LEN | msa.MSA_DEVERR_BAD_PAGE
    kv = values(cache)
    rows = []
    for b, skip in ((1, 1), (2, 0)):
        t = np.arange(lengths[b])
        rows.append([places(pt[b].numpy().clip(0, len(kv[0]) - 1), t[t // BK != skip])] * 2)
    check_rows(Q[1:], kv, rows, (O[1:], LSE[1:]))
    assert np.all(O[0] == 0) and np.all(np.isneginf(LSE[0]))
    # a page of another sequence's length past the table
    assert run_dense(msa, Q, cache, pt, [200, BK * pt.shape[1] + 1, 300])[2] & msa.MSA_DEVERR_BAD_LEN


def test_workspace_serves_calls_of_all_shapes(msa):
    """One zero-filled workspace, calls of several shapes and kinds in turn without clearing."""
    ws = torch.zeros(msa.msa_attn_decode_q8_workspace_size(64, 8), dtype=torch.uint8, device="cuda")
    for seed, (lengths, Hkv, G, w) in enumerate([([9000], 1, 4, 0), ([5000, 100], 8, 6, 0), ([800] * 64, 2, 2, 0), ([9000], 1, 4, 3000),
                                                 ([30000], 2, 1, 0), ([700] * 9, 4, 8, 200)]):
        Q, cache, pt = dense_case(msa, lengths, Hkv, G, seed)
        got = run_dense(msa, Q, cache, pt, lengths, w, 0, ws=ws, zeroed=True)
        check_dense(Q, cache, pt, lengths, got[:2], w)
        k = min(8, pt.shape[1])
        n = torch.full((len(lengths) * Hkv,), k, dtype=torch.int32, device="cuda").clamp(max=min(-(-L // BK) for L in lengths))
        sp = pt[:, :k].repeat_interleave(Hkv, 0).contiguous().cuda()
        a = run_sparse(msa, Q, cache, sp, n, torch.full_like(n, 64), zeroed=True, ws=ws)
        b = run_sparse(msa, Q, cache, sp, n, torch.full_like(n, 64))
        assert np.array_equal(a[0], b[0]) and a[2] == 0


def test_captured_and_on_another_stream(msa):
    lengths = [3000, 100, 0, 777]
    Q, cache, pt = dense_case(msa, lengths, 4, 6, 11)
    want = run_dense(msa, Q, cache, pt, lengths)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run_dense(msa, Q, cache, pt, lengths)
    torch.cuda.synchronize()
    assert np.array_equal(want[0], got[0])
    O = torch.zeros(4, 24, D, dtype=torch.bfloat16, device="cuda")
    LSE = torch.zeros(4, 24, device="cuda")
    ws = torch.zeros(msa.msa_attn_decode_q8_workspace_size(4, 4), dtype=torch.uint8, device="cuda")
    ptc, L = pt.cuda(), dev(lengths, torch.int32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_dense_attn_decode_q8(Q, cache, ptc, L, O, LSE, ws)
    for _ in range(3):
        O.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(O), want[0])
    L.copy_(dev([100, 3000 - 2900, 5, 0], torch.int32))   # other lengths, the same graph
    graph.replay()
    torch.cuda.synchronize()
    other = run_dense(msa, Q, cache, pt, [100, 100, 5, 0])
    assert np.array_equal(host(O), other[0])


def test_step_over_the_cache(msa):
    """Tokens through msa_plan_step's slots into the cache, then decode_step_q8, against decode_step over the expanded pages:
    the same selection, and attention over the same values."""
    from workloads import DecodeWorkload, MSAShape, decode_inputs
    wl = DecodeWorkload("q8_step", lengths=(1, 700, 3000, 129), shape=MSAShape(k=4), seed=78)
    inp = decode_inputs(wl, device="cuda:0")
    P, Hkv = inp["K_pool"].shape[:2]
    cache = msa.q8_cache(P, Hkv, "cuda")
    for b, L in enumerate(wl.lengths):
        t = torch.arange(L, device="cuda")
        page = inp["seq_pt"][b].long()[t // BK]
        msa.msa_cache_append_q8(inp["K_pool"][page, :, t % BK], inp["V_pool"][page, :, t % BK], page * BK + t % BK, cache)
    out = [torch.empty(P, Hkv, BK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    msa.msa_cache_expand_q8(cache, torch.arange(P, dtype=torch.int32, device="cuda"), *out)
    # E4M3 keeps four bits: half a step is 2^-4 of a value, and 2^-10 of the block's scale below its normal range
    for o, x, s in zip(out, (inp["K_pool"], inp["V_pool"]), (cache.K_scales, cache.V_scales)):
        for b, L in enumerate(wl.lengths):
            t = torch.arange(L, device="cuda")
            page = inp["seq_pt"][b].long()[t // BK]
            a, w = o[page, :, t % BK].float(), x[page, :, t % BK].float()
            # (a value may have been rounded under a smaller scale before)
            step = torch.pow(2.0, s[page].float() - 127)[..., None]
            assert bool(((a - w).abs() <= 2 * (w.abs() * 2 ** -4 + step * 2.0 ** -10)).all())
    got = msa.decode_step_q8(inp, cache, 4)
    want = msa.decode_step({**inp, "K_pool": out[0], "V_pool": out[1]}, 4)
    torch.cuda.synchronize()
    assert int(got["dev_err"].item()) == 0
    assert torch.equal(got["sel"], want["sel"]) and torch.equal(got["pt"], want["pt"])
    size = float(out[1].abs().max())
    assert float((got["O"].float() - want["O"].float()).abs().max()) <= size * 2.0 ** -6   # two roundings of P and O each
    assert float((got["LSE"] - want["LSE"]).abs().max()) <= 1e-4
