"""Attention through a sliding window with sinks on the GPU: one query per sequence over bf16 pages, and many queries over
contiguous tensors and pages, against 64-bit definitions."""
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


def dev(a):
    return torch.as_tensor(np.asarray(a)).to(device="cuda", dtype=torch.int32)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def paged(lengths, Hkv, seed, extra=3):
    """Pools of normal values and a shuffled page table for sequences of these lengths."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-L // BK) for L in lengths]
    pool = sum(per) + extra
    ids = torch.randperm(pool, generator=g).int()
    pt = torch.full((len(lengths), max(max(per), 1)), -1, dtype=torch.int32)
    for b, n in enumerate(per):
        pt[b, :n] = ids[sum(per[:b]):sum(per[:b + 1])]
    K, V = (torch.randn(pool, Hkv, BK, D, generator=g).bfloat16() for _ in range(2))
    return g, K, V, pt


# ---------------------------------------------------------------------------
# one query per sequence
# ---------------------------------------------------------------------------

def run_decode(msa, Q, K, V, pt, lengths, window, sinks, scale=0.0, ws=None, zeroed=False):
    B, Hq, _ = Q.shape
    O = torch.full((B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((B, Hq), 7.0, device="cuda")
    if ws is None:
        ws = torch.zeros(msa.msa_window_attn_decode_workspace_size(B, K.shape[1]), dtype=torch.uint8, device="cuda")
    e = dev([0])
    msa.msa_window_attn_decode(Q, K, V, pt.cuda(), dev(lengths), O, LSE, ws, window=window, sinks=sinks, softmax_scale=scale,
                               dev_err=e, scratch_zeroed=zeroed)
    return host(O), LSE.double().cpu().numpy(), int(e.item())


def check_decode(Q, K, V, pt, lengths, window, sinks, got, scale=1 / math.sqrt(D), skip=()):
    q, k, v = host(Q), host(K), host(V)
    Hkv = k.shape[1]
    G = q.shape[1] // Hkv
    for b, L in enumerate(lengths):
        t = ref.seen(L - 1, window, sinks)
        page = pt[b].numpy()[t // BK]
        ok = (page >= 0) & (page < len(k))
        page, t = page[ok], t[ok]
        for g in range(Hkv):
            h = slice(g * G, (g + 1) * G)
            ref.check(got[0][b, h], got[1][b, h], ref.attend(q[b, h], k[page, g, t % BK], v[page, g, t % BK], scale), ref.HALF["bf16"])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (17, 4), (128, 0), (130, 129), (2048, 4), (1 << 30, 0)])
@pytest.mark.parametrize("lengths,Hkv,G", [([1, 2, 16, 130, 0, 700, 3000], 2, 6), ([12000], 1, 8), ([400] * 70, 8, 1), ([5000] * 3, 3, 5)])
def test_decode(msa, window, sinks, lengths, Hkv, G):
    g, K, V, pt = paged(lengths, Hkv, window % 1000 + sinks + G)
    Q = (torch.randn(len(lengths), Hkv * G, D, generator=g) * 1.5).bfloat16().cuda()
    K, V = K.cuda(), V.cuda()
    got = run_decode(msa, Q, K, V, pt, lengths, window, sinks)
    assert got[2] == 0
    check_decode(Q, K, V, pt, lengths, window, sinks, got)
    again = run_decode(msa, Q, K, V, pt, lengths, window, sinks)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


def test_decode_strides_scale_and_unseen_slots(msa):
    lengths, window, sinks = [300, 1000, 129], 140, 3
    g, K, V, pt = paged(lengths, 2, 1)
    Q = (torch.randn(3, 2 * 12, D, generator=g)).bfloat16().cuda()[:, ::2]
    wide = torch.full((2, K.shape[0], 3, BK, 2 * D), math.nan, dtype=torch.bfloat16, device="cuda")
    views = wide[0, :, 1:, :, :D], wide[1, :, 1:, :, :D]
    for view, x in zip(views, (K, V)):
        view.copy_(x)
    want = run_decode(msa, Q.contiguous(), K.cuda(), V.cuda(), pt, lengths, window, sinks, scale=0.3)
    for b, L in enumerate(lengths):
        see = set(ref.seen(L - 1, window, sinks).tolist())
        for t in range(-(-L // BK) * BK):
            if t not in see:
                for x in views:
                    x[pt[b, t // BK].item(), :, t % BK] = math.nan
    got = run_decode(msa, Q, *views, pt, lengths, window, sinks, scale=0.3)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    check_decode(Q, K, V, pt, lengths, window, sinks, got, scale=0.3)


def test_decode_bad_lengths_and_pages(msa):
    lengths = [300, 1000, 500]
    g, K, V, pt = paged(lengths, 2, 2)
    pt[1, 7], pt[2, 0], pt[1, 3] = K.shape[0], -1, -9      # the last one lies before the window and is not looked at
    Q = torch.randn(3, 4, D, generator=g).bfloat16().cuda()
    got = run_decode(msa, Q, K.cuda(), V.cuda(), pt, [-3, 1000, 500], 300, 5)
    assert got[2] == msa.MSA_DEVERR_BAD_LEN | msa.MSA_DEVERR_BAD_PAGE
    assert np.all(got[0][0] == 0) and np.all(np.isneginf(got[1][0]))
    check_decode(Q[1:], K, V, pt[1:], lengths[1:], 300, 5, (got[0][1:], got[1][1:]))


def test_decode_as_the_last_row_of_a_prefill(msa):
    """One query at the end of every sequence: as msa_window_attn_prefill's over the same pages, up to the rounding of P."""
    lengths = [1, 128, 900, 4000]
    g, K, V, pt = paged(lengths, 2, 3)
    Q = torch.randn(4, 12, D, generator=g).bfloat16().cuda()
    a = run_decode(msa, Q, K.cuda(), V.cuda(), pt, lengths, 500, 130)
    b = run_prefill(msa, Q[:, None], K.cuda(), V.cuda(), 500, 130, pt, [L - 1 for L in lengths])
    assert np.abs(a[0] - b[0][:, 0]).max() <= 2.0 ** -7 * np.abs(a[0]).max() + 2.0 ** -8 * 5
    assert np.abs(a[1] - b[1][:, 0]).max() <= 1e-4


# ---------------------------------------------------------------------------
# many queries
# ---------------------------------------------------------------------------

def run_prefill(msa, Q, K, V, window, sinks, pt=None, pos=None, scale=0.0):
    B, S, Hq, _ = Q.shape
    O = torch.full((B, S, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((B, S, Hq), 7.0, device="cuda")
    e = dev([0])
    msa.msa_window_attn_prefill(Q, K, V, O, LSE, window=window, sinks=sinks, softmax_scale=scale, dev_err=e,
                                seq_pt=None if pt is None else pt.cuda(), q_pos=None if pos is None else dev(pos))
    return host(O), LSE.double().cpu().numpy(), int(e.item())


def check_prefill(Q, K, V, window, sinks, got, pt=None, pos=None, scale=1 / math.sqrt(D), rows=None):
    q, k, v = host(Q), host(K), host(V)
    B, S, Hq, _ = q.shape
    Hkv = k.shape[2] if pt is None else k.shape[1]
    G = Hq // Hkv
    for b in range(B):
        if pt is not None:
            page = pt[b].numpy()
            n = -(-(pos[b] + S) // BK)
            live = np.repeat((page[:n] >= 0) & (page[:n] < len(k)), BK)
            kb, vb = (x[page[:n].clip(0, len(k) - 1)].transpose(0, 2, 1, 3).reshape(-1, Hkv, D) for x in (k, v))
        for s in (range(S) if rows is None else rows):
            t = ref.seen(s + (pos[b] if pos is not None else 0), window, sinks)
            for g in range(Hkv):
                h = slice(g * G, (g + 1) * G)
                if pt is None:
                    kk, vv = k[b, t, g], v[b, t, g]
                else:
                    kk, vv = kb[t[live[t]], g], vb[t[live[t]], g]
                ref.check(got[0][b, s, h], got[1][b, s, h], ref.attend(q[b, s, h], kk, vv, scale), ref.HALF["bf16"])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (30, 4), (128, 0), (129, 128), (200, 140), (1 << 30, 5)])
@pytest.mark.parametrize("B,S,Hkv,G", [(1, 1, 1, 1), (2, 5, 2, 6), (1, 130, 1, 3), (3, 129, 2, 8), (1, 700, 2, 6), (2, 400, 1, 7), (1, 600, 2, 1)])
def test_prefill(msa, window, sinks, B, S, Hkv, G):
    g = torch.Generator().manual_seed(S + G)
    Q = (torch.randn(B, S, Hkv * G, D, generator=g) * 1.5).bfloat16().cuda()
    K, V = (torch.randn(B, S, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    got = run_prefill(msa, Q, K, V, window, sinks)
    assert got[2] == 0
    check_prefill(Q, K, V, window, sinks, got, rows=None if S < 200 else [0, 1, 20, 21, 41, 42, 43, 63, 64, 126, 127, 128, 129, 199, 200, 255, 256, 300, S - 1])
    again = run_prefill(msa, Q, K, V, window, sinks)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (300, 130), (1000, 0), (1 << 30, 0)])
@pytest.mark.parametrize("pos,S,Hkv,G", [([0], 1, 1, 4), ([0, 1, 127, 128, 129], 4, 2, 6), ([1000, 3, 500], 150, 1, 8), ([2000], 300, 2, 5),
                                         ([700] * 20, 3, 8, 6)])
def test_chunk(msa, window, sinks, pos, S, Hkv, G):
    g, K, V, pt = paged([p + S for p in pos], Hkv, S + window % 100)
    Q = (torch.randn(len(pos), S, Hkv * G, D, generator=g) * 1.5).bfloat16().cuda()
    K, V = K.cuda(), V.cuda()
    got = run_prefill(msa, Q, K, V, window, sinks, pt, pos)
    assert got[2] == 0
    check_prefill(Q, K, V, window, sinks, got, pt, pos, rows=None if S < 20 else [0, 1, 15, 16, 20, 21, 42, 99, S - 1])


def test_chunk_equals_prefill(msa):
    """A chunk from position 0 over pages, and chunks one after another, give what the contiguous call gives."""
    S, Hkv, G = 1000, 2, 6
    g, K, V, pt = paged([S], Hkv, 9)
    K, V = K.cuda(), V.cuda()
    Q = torch.randn(1, S, Hkv * G, D, generator=g).bfloat16().cuda()
    flat = [x[pt[0].cuda().long()].transpose(1, 2).reshape(1, -1, Hkv, D)[:, :S].contiguous() for x in (K, V)]
    want = run_prefill(msa, Q, *flat, 300, 10)
    got = run_prefill(msa, Q, K, V, 300, 10, pt, [0])
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    part = run_prefill(msa, Q[:, 500:], K, V, 300, 10, pt, [500])
    assert np.abs(part[0] - want[0][:, 500:]).max() <= 2.0 ** -6 and np.abs(part[1] - want[1][:, 500:]).max() <= 1e-4


def test_whole_window_is_causal_attention(msa):
    """A window of the whole length, against the framework's dense prefill."""
    g = torch.Generator().manual_seed(10)
    Q = torch.randn(1, 900, 12, D, generator=g).bfloat16().cuda()
    K, V = (torch.randn(1, 900, 2, D, generator=g).bfloat16().cuda() for _ in range(2))
    got = run_prefill(msa, Q, K, V, 900, 0)
    want = msa.dense_prefill_layer({"Q": Q, "K": K, "V": V})
    assert np.abs(got[0] - host(want["O"])).max() <= 2.0 ** -6 and np.abs(got[1] - host(want["LSE"])).max() <= 1e-4


def test_prefill_strides_and_large_scores(msa):
    g = torch.Generator().manual_seed(11)
    wide = torch.randn(2, 260, 3 * 8, D, generator=g).bfloat16().cuda()
    Q, K, V = wide[:, ::2, :16:2], wide[:, 1::2, 16:20:2], wide[:, 1::2, 20:24:2]
    got = run_prefill(msa, Q, K, V, 50, 2, scale=0.2)
    check_prefill(Q, K, V, 50, 2, got, scale=0.2)
    # equal keys have equal weights, however large the scores
    for size in (1e4, 1e9, 1e15):
        Q = torch.full((1, 200, 4, D), size, dtype=torch.bfloat16, device="cuda")
        K = torch.ones(1, 200, 1, D, dtype=torch.bfloat16, device="cuda")
        V = torch.randn(1, 200, 1, D, generator=g).bfloat16().cuda()
        O, LSE, e = run_prefill(msa, Q, K, V, 64, 4)
        v = host(V)[0, :, 0]
        for i in (0, 5, 63, 64, 199):
            x = v[ref.seen(i, 64, 4)]
            assert np.all(np.abs(O[0, i] - x.mean(0)) <= np.abs(x.mean(0)) * 2.0 ** -8 + np.abs(x).mean(0) * 2.0 ** -8)


def test_chunk_bad_positions_and_pages(msa):
    S, pos = 40, [-1, 300, 500, 600]
    g, K, V, pt = paged([640] * 4, 2, 12)
    pt[1, 0], pt[1, 2] = -1, K.shape[0] + 7
    K, V = K.cuda(), V.cuda()
    Q = torch.randn(4, S, 12, D, generator=g).bfloat16().cuda()
    O, LSE, e = run_prefill(msa, Q, K, V, 100, 3, pt, [-1, 300, 500, 601])
    assert e == msa.MSA_DEVERR_BAD_LEN | msa.MSA_DEVERR_BAD_PAGE
    for b in (0, 3):
        assert np.all(O[b] == 0) and np.all(np.isneginf(LSE[b]))
    check_prefill(Q[1:3], K, V, 100, 3, (O[1:3], LSE[1:3]), pt[1:3], pos[1:3])


@pytest.mark.parametrize("pos,S", [([0, 5, 100, 127], 1), ([300, 61, 0, 90], 40), ([1000, 127, 64, 63], 130)])
def test_chunk_anything_behind_the_last_token(msa, pos, S):
    g, K, V, pt = paged([p + S for p in pos], 2, 14)
    Q = torch.randn(4, S, 12, D, generator=g).bfloat16().cuda()
    K, V = K.cuda(), V.cuda()
    for window, sinks in ((100, 3), (1 << 30, 0)):
        want = run_prefill(msa, Q, K, V, window, sinks, pt, pos)
        wild = [x.clone() for x in (K, V)]
        for b, p in enumerate(pos):
            for t in range(p + S, -(-(p + S) // BK) * BK):
                for x, v in zip(wild, (math.nan, -math.inf if t % 2 else math.nan)):
                    x[pt[b, t // BK].item(), :, t % BK] = v
        got = run_prefill(msa, Q, *wild, window, sinks, pt, pos)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_graphs_and_streams(msa):
    lengths, S = [700, 300], 20
    g, K, V, pt = paged([L + S for L in lengths], 2, 13)
    K, V, ptc = K.cuda(), V.cuda(), pt.cuda()
    Q = torch.randn(2, S, 12, D, generator=g).bfloat16().cuda()
    want = run_prefill(msa, Q, K, V, 100, 3, pt, lengths)
    dec = run_decode(msa, Q[:, -1].contiguous(), K, V, pt, [L + S for L in lengths], 100, 3)
    O, O1 = torch.zeros(2, S, 12, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 12, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(msa.msa_window_attn_decode_workspace_size(2, 2), dtype=torch.uint8, device="cuda")
    pos, n, last = dev(lengths), dev([L + S for L in lengths]), Q[:, -1].contiguous()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_window_attn_prefill(Q, K, V, O, None, window=100, sinks=3, seq_pt=ptc, q_pos=pos)
        msa.msa_window_attn_decode(last, K, V, ptc, n, O1, None, ws, window=100, sinks=3, scratch_zeroed=True)
    for _ in range(3):
        O.fill_(5)
        O1.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(O), want[0]) and np.array_equal(host(O1), dec[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    O.fill_(5)
    torch.cuda.synchronize()
    msa.msa_window_attn_prefill(Q, K, V, O, None, window=100, sinks=3, seq_pt=ptc, q_pos=pos, stream=s)
    s.synchronize()
    assert np.array_equal(host(O), want[0])


def test_calls_and_graphs_share_a_workspace(msa):
    """One zero-filled workspace, 8-bit and bf16 calls of several shapes in turn, eager and from two captured graphs."""
    g, K, V, pt = paged([3000, 129, 0, 7000], 2, 15)
    K, V, ptc, n = K.cuda(), V.cuda(), pt.cuda(), dev([3000, 129, 0, 7000])
    Q = torch.randn(4, 12, D, generator=g).bfloat16().cuda()
    cache = msa.q8_cache(K.shape[0], 2, "cuda")
    page = torch.arange(K.shape[0] * BK, device="cuda")
    msa.msa_cache_append_q8(*(x.transpose(1, 2).reshape(-1, 2, D).contiguous() for x in (K, V)), page, cache)
    ws = torch.zeros(msa.msa_window_attn_decode_workspace_size(4, 2), dtype=torch.uint8, device="cuda")
    out = [torch.zeros(4, 12, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    sparse = ptc[[0, 0, 3, 3], :20].contiguous()                                     # [2 * Hkv, 20]

    def all_bf16(o, ws):
        msa.msa_window_attn_decode(Q, K, V, ptc, n, o, None, ws, window=1 << 30, scratch_zeroed=True)

    def short(o, ws):
        msa.msa_window_attn_decode(Q[1:], K, V, ptc[1:], n[1:], o[1:], None, ws, window=4000, sinks=200, scratch_zeroed=True)

    def all_q8(o, ws):
        msa.msa_dense_attn_decode_q8(Q, cache, ptc, n, o, None, ws, scratch_zeroed=True)

    def some_q8(o, ws):
        msa.msa_sparse_attn_decode_q8(Q[:2], cache, sparse, dev([20, 7, 20, 20]), dev([128] * 4), o[:2], None, ws, scratch_zeroed=True)

    calls = (all_bf16, short, all_q8, some_q8)
    want = []
    for call in calls:
        o = torch.zeros_like(out[0])
        call(o, torch.zeros_like(ws))
        want.append(host(o))
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (2, 0, 2, 1, 3, 0)):
        for i in order:
            out[i].zero_()
            calls[i](out[i], ws)
            assert np.array_equal(host(out[i]), want[i])
    graphs = []
    for i, j in ((2, 1), (0, 2)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            calls[i](out[i], ws)
            calls[j](out[j], ws)
    for _ in range(2):
        for graph, pair in zip(graphs, ((2, 1), (0, 2))):
            for o in out:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for i in pair:
                assert np.array_equal(host(out[i]), want[i])


def test_few_tiles_many_launches(msa):
    """Draft tokens over pools whose first reads miss every cache: a K/V block that lands later than the other slot's blocks
    behind it is waited for all the same.  (One launch in some 20,000 had run into the wait's limit.)"""
    B, S, per = 8, 4, 400
    g = torch.Generator(device="cuda").manual_seed(16)
    pools = [[torch.randn(B * per, 8, BK, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2)] for _ in range(2)]
    pt = torch.randperm(B * per, generator=g, device="cuda").int().view(B, per)
    Q, pos, e = torch.randn(B, S, 48, D, generator=g, device="cuda").bfloat16(), dev([per * BK - S] * B), dev([0])
    out = [(torch.empty_like(Q), torch.empty(B, S, 48, device="cuda")) for _ in range(2)]
    want = []
    for i in range(40000):
        (K, V), (O, LSE) = pools[i % 2], out[i % 2]
        msa.msa_window_attn_prefill(Q, K, V, O, LSE, window=2048, sinks=4, seq_pt=pt, q_pos=pos, dev_err=e)
        if i < 2:
            want.append((O.clone(), LSE.clone()))
        if i % 4000 >= 3998:
            assert int(e.item()) == 0 and torch.equal(O, want[i % 2][0]) and torch.equal(LSE, want[i % 2][1])


# ---------------------------------------------------------------------------
# more tiles than SMs: a CTA works on pairs of tiles, one after another
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("window,sinks", [(1, 0), (30, 4), (129, 128), (200, 140), (1 << 30, 5)])
@pytest.mark.parametrize("B,S,Hkv,G", [(3, 500, 8, 6), (16, 130, 8, 1), (2, 700, 8, 8), (4, 333, 8, 7), (40, 21, 4, 6), (40, 22, 4, 6), (5, 200, 8, 3),
                                       (3, 270, 16, 5), (9, 200, 8, 2), (8, 150, 8, 4), (200, 1, 1, 6)])
def test_many_tiles(msa, window, sinks, B, S, Hkv, G):
    g = torch.Generator().manual_seed(S + G)
    Q = (torch.randn(B, S, Hkv * G, D, generator=g) * 1.5).bfloat16().cuda()
    K, V = (torch.randn(B, S, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    got = run_prefill(msa, Q, K, V, window, sinks)
    assert got[2] == 0
    nq = 128 // G
    rows = sorted({r for r in (0, nq - 1, nq, 2 * nq - 1, 2 * nq, 63, 64, 128, 129, 199, S - nq, S - 1) if 0 <= r < S})
    few = [0, B - 1]                             # (sequences that are checked; the others against the same one alone)
    check_prefill(Q[few], K[few], V[few], window, sinks, (got[0][few], got[1][few]), rows=rows)
    b = B // 2
    one = run_prefill(msa, Q[b:b + 1], K[b:b + 1], V[b:b + 1], window, sinks)
    # (each rounds P and O to bf16, 2^-8 of the largest value at most)
    assert np.abs(one[0][0] - got[0][b]).max() <= 4 * 2.0 ** -8 * float(V[b].abs().max()) and np.abs(one[1][0] - got[1][b]).max() <= 1e-4
    again = run_prefill(msa, Q, K, V, window, sinks)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


@pytest.mark.parametrize("S,Hkv,G", [(40, 8, 6), (21, 8, 6), (70, 8, 8), (150, 8, 2)])
@pytest.mark.parametrize("window,sinks", [(100, 3), (1 << 30, 0)])
def test_many_tiles_over_pages(msa, S, Hkv, G, window, sinks):
    """With positions and pages that are none, and anything in the slots behind the last tokens."""
    pos = [0, 300, -1, 61, 127, 500, 64, 1 << 20, 10, 333, 700, 128, 5, 90, 211, 400, 1, 2, 3, 255, 256, 257]
    g, K, V, pt = paged([(p + S if 0 <= p < 1000 else 1) for p in pos], Hkv, S)
    pt[1, 0], pt[5, 2], pt[9, 1] = -1, K.shape[0] + 7, -5
    Q = torch.randn(len(pos), S, Hkv * G, D, generator=g).bfloat16().cuda()
    for b, p in enumerate(pos):
        if 0 <= p < 1000:
            for t in range(p + S, -(-(p + S) // BK) * BK):
                if 0 <= pt[b, t // BK] < len(K):
                    K[pt[b, t // BK], :, t % BK], V[pt[b, t // BK], :, t % BK] = math.nan, -math.inf if t % 2 else math.nan
    K, V = K.cuda(), V.cuda()
    got = run_prefill(msa, Q, K, V, window, sinks, pt, pos)
    assert got[2] == msa.MSA_DEVERR_BAD_LEN | msa.MSA_DEVERR_BAD_PAGE
    bad = [b for b, p in enumerate(pos) if not 0 <= p < 1000]
    assert (got[0][bad] == 0).all() and np.isneginf(got[1][bad]).all()
    few = [b for b in range(0, len(pos), 3) if b not in bad] + [1, 5]
    check_prefill(Q[few], K, V, window, sinks, (got[0][few], got[1][few]), pt[few], [pos[b] for b in few],
                  rows=sorted({0, min(15, S - 1), 20, min(21, S - 1), S - 1}))


def test_many_tiles_large_scores_and_rising_ones(msa):
    g = torch.Generator().manual_seed(18)
    V = torch.randn(1, 900, 8, D, generator=g).bfloat16().cuda()
    v = host(V)[0]
    for size in (1e4, 1e9, 1e15):                # equal keys have equal weights, however large the scores
        Q = torch.full((1, 900, 32, D), size, dtype=torch.bfloat16, device="cuda")
        K = torch.ones(1, 900, 8, D, dtype=torch.bfloat16, device="cuda")
        O, LSE, e = run_prefill(msa, Q, K, V, 64, 4)
        for i in (0, 5, 63, 64, 500, 899):
            for h in (0, 31):
                x = v[ref.seen(i, 64, 4), h // 4]
                assert np.all(np.abs(O[0, i, h] - x.mean(0)) <= np.abs(x.mean(0)) * 2.0 ** -8 + np.abs(x).mean(0) * 2.0 ** -8)
    # every block's scores are far above those of the block before: the running maximum moves and O is rescaled each time
    Q = torch.randn(1, 900, 32, D, generator=g).abs().bfloat16().cuda()
    K = (torch.rand(1, 900, 8, D, generator=g) * (1 + torch.arange(900)[None, :, None, None] // 64)).bfloat16().cuda()
    for K in (K, K.flip(1).contiguous()):
        got = run_prefill(msa, Q, K, V, 1 << 30, 0)
        check_prefill(Q, K, V, 1 << 30, 0, got, rows=[0, 20, 21, 63, 64, 130, 500, 899])
