"""The serving step around the paged cache on the GPU: page tables and slots, head
norm with rotation, the 4-bit store, decode attention over it, and a run of all
of them, against 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu
BK = 128


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def dev(a, dtype=None):
    return torch.as_tensor(np.asarray(a)).to(device="cuda", dtype=dtype)


def i32(a):
    return dev(a, torch.int32)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# page tables and slots
# ---------------------------------------------------------------------------

def run_plan(msa, L, n, seq_pt, free, count, N, num_pages, in_place=False):
    t = {"L": i32(L), "n": i32(n), "pt": i32(seq_pt), "free": i32(free), "count": i32([count])}
    o = msa.plan_buffers(len(L), N, "cuda")
    for x in o.values():
        x.fill_(-77)
    if in_place:
        o["seq_len_out"], o["free_count_out"] = t["L"], t["count"]
    e = err_word()
    msa.msa_plan_step(t["L"], t["n"], t["pt"], t["free"], t["count"], *[o[k] for k in (
        "seq_len_out", "free_count_out", "cu", "tok_slot", "tok_pos", "tok_seq")], num_pages=num_pages, dev_err=e)
    got = {k: v.cpu().numpy().astype(np.int64) for k, v in o.items()}
    got["seq_pt"], got["err"] = t["pt"].cpu().numpy(), int(e.item())
    return got


def check_plan(got, want):
    for k in ("seq_len_out", "cu", "tok_slot", "tok_pos", "tok_seq", "seq_pt"):
        assert np.array_equal(got[k], want[k]), k
    assert got["free_count_out"][0] == want["free_count_out"] and got["err"] == want["err"]


def plan_case(B, max_pages, lens, new, pad, seed, short=0):
    """Lengths, tables over shuffled page ids and a stack of the rest, less ``short`` pages."""
    r = np.random.default_rng(seed)
    L = np.array([lens(r) for _ in range(B)], dtype=np.int64)
    n = np.array([min(new(r), max_pages * BK - l) for l in L], dtype=np.int64)
    need = sum(-(-(a + b) // BK) for a, b in zip(L, n))
    pool = need + 7
    ids = r.permutation(pool)
    pt, at = np.full((B, max_pages), -1, dtype=np.int64), 0
    for b in range(B):
        have = -(-L[b] // BK)
        pt[b, :have] = ids[at:at + have]
        at += have
    free = np.full(pool, -5, dtype=np.int64)
    free[:pool - at] = ids[at:]
    return L, n, pt, free, pool - at - 7 - short, int(n.sum()) + pad, pool


PLANS = {
    "one": lambda: plan_case(1, 4, lambda r: 0, lambda r: 1, 0, 1),
    "decode": lambda: plan_case(8, 512, lambda r: 60001, lambda r: 1, 0, 2),
    "edges": lambda: plan_case(40, 6, lambda r: int(r.choice([0, 1, 127, 128, 129, 256])),
                               lambda r: int(r.choice([0, 1, 127, 128, 129, 400])), 5, 3),
    "many": lambda: plan_case(4096, 5, lambda r: int(r.integers(0, 300)), lambda r: int(r.integers(0, 9)), 1000, 4),
    "prompts": lambda: plan_case(33, 200, lambda r: int(r.integers(0, 9000)), lambda r: int(r.integers(0, 9000)), 311, 5),
    "b1025": lambda: plan_case(1025, 9, lambda r: int(r.integers(0, 500)), lambda r: int(r.integers(0, 40)), 0, 6),
    "idle": lambda: plan_case(5, 3, lambda r: 17, lambda r: 0, 4, 7),
    "out_of_pages": lambda: plan_case(60, 20, lambda r: int(r.integers(0, 900)), lambda r: int(r.integers(0, 300)), 9, 8, short=25),
    "out_of_pages_many": lambda: plan_case(3000, 20, lambda r: int(r.integers(0, 900)), lambda r: int(r.integers(0, 30)), 0, 9,
                                           short=300),
}


@pytest.mark.parametrize("name", PLANS)
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_step(msa, name, in_place):
    c = PLANS[name]()
    check_plan(run_plan(msa, *c, in_place=in_place), ref.plan(*c))


def test_plan_step_bad_requests(msa):
    """A bad length, one past the table, rows past N, bad page ids and a bad stack height: named in the error word,
    the other requests served."""
    L, n, pt, free, count, N, pool = plan_case(12, 8, lambda r: int(r.integers(1, 500)), lambda r: 200, 0, 11)
    L[2], n[3], L[5], n[5] = -1, -4, 900, 200
    check_plan(run_plan(msa, L, n, pt, free, count, N, pool), ref.plan(L, n, pt, free, count, N, pool))
    N = int(np.maximum(n, 0)[:9].sum()) + 50                     # request 9's rows pass the end
    check_plan(run_plan(msa, L, n, pt, free, count, N, pool), ref.plan(L, n, pt, free, count, N, pool))
    pt[0, :] = pool + 3
    free[count - 2] = -9
    check_plan(run_plan(msa, L, n, pt, free, count, N, pool), ref.plan(L, n, pt, free, count, N, pool))
    for bad in (-3, len(free) + 5):
        check_plan(run_plan(msa, L, n, pt, free, bad, N, pool), ref.plan(L, n, pt, free, bad, N, pool))


def test_plan_step_without_rows_or_requests(msa):
    L, n, pt, free, count, _, pool = PLANS["edges"]()
    n = n * 0
    check_plan(run_plan(msa, L, n, pt, free, count, 0, pool), ref.plan(L, n, pt, free, count, 0, pool))
    none = np.zeros(0, dtype=np.int64)
    c = (none, none, np.zeros((0, 3), dtype=np.int64), free, count, 6, pool)
    check_plan(run_plan(msa, *c), ref.plan(*c))


@pytest.mark.parametrize("B,max_pages,seed", [(1, 3, 1), (7, 40, 2), (200, 5, 3), (4096, 4, 4), (64, 700, 5)])
def test_release_pages(msa, B, max_pages, seed):
    r = np.random.default_rng(seed)
    L = r.integers(0, max_pages * BK + 1, B)
    done = (r.random(B) < 0.6).astype(np.int64) * r.integers(1, 9, B)
    pt = r.permutation(B * max_pages).reshape(B, max_pages)
    if B == 200:
        L[3], L[9], done[3], done[9] = -2, max_pages * BK + 1, 1, 1
    for cap in (B * max_pages + 9, B * max_pages // 3):          # the second overflows
        free = r.permutation(cap)
        want = ref.release(L, done, pt, free, 5)
        t = i32(L), i32(done), i32(pt), i32(free), i32([5])
        out, cnt, e = torch.full_like(t[0], -7), i32([-1]), err_word()
        msa.msa_release_pages(*t, out, cnt, dev_err=e)
        assert np.array_equal(out.cpu(), want["seq_len_out"]) and int(cnt) == want["free_count_out"]
        assert np.array_equal(t[3].cpu(), want["free_pages"]) and int(e) == want["err"]
        msa.msa_release_pages(*t, t[0], t[4])                    # in place
        assert np.array_equal(t[0].cpu(), want["seq_len_out"]) and int(t[4]) == want["free_count_out"]


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------

def rope_case(N, Hq, Hkv, D, rot, seed, far=131072, wdtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = (1.3 * torch.randn(N, Hq + 2 * Hkv, D, generator=g, device="cuda")).bfloat16()
    w = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(wdtype) for _ in range(2)]
    pos = torch.randint(0, far, (N,), generator=g, device="cuda", dtype=torch.int32)
    f = (5e6 ** (-torch.arange(0, rot, 2, device="cuda").double() / max(rot, 1))).float() if rot else None
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], w[0], w[1], pos, f


def check_rope(got, x, w, pos, f, interleaved, eps=1e-6):
    """fp32 sums, root and products (2^-17 at worst of a norm over 128 values) and the sines' 2^-21, then bf16's 2^-8."""
    y, size = ref.norm_rope(ref.f64(x), None if w is None else ref.f64(w), ref.f64(pos),
                            None if f is None else ref.f64(f), eps, interleaved)
    err = np.abs(ref.f64(got) - y)
    assert (err <= 2.0 ** -8 * np.abs(y) + 2.0 ** -16 * size + 1e-30).all(), err.max()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,Hq,Hkv,D,rot", [(1, 1, 1, 128, 128), (8, 48, 8, 128, 128), (131, 6, 2, 128, 64), (77, 5, 3, 128, 16),
                                            (300, 32, 8, 64, 32), (33, 9, 1, 64, 64), (5, 7, 2, 64, 16), (6000, 12, 4, 128, 96),
                                            (64, 8, 8, 128, 0)])
def test_norm_rope(msa, N, Hq, Hkv, D, rot, interleaved):
    Q, K, V, wq, wk, pos, f = rope_case(N, Hq, Hkv, D, rot, 5 * N + rot)
    Qo, Ko = torch.empty(N, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty_like(K, memory_format=torch.contiguous_format)
    msa.msa_qk_norm_rope(Q, K, pos, f, Qo, Ko, q_weight=wq, k_weight=wk, interleaved=interleaved)
    check_rope(Qo, Q, wq, pos, f, interleaved)
    check_rope(Ko, K, wk, pos, f, interleaved)
    # into pages, with the values, and Q in place
    P = N // BK + 2
    slots = torch.randperm(P * BK, device="cuda")[:N]
    Kp, Vp = (torch.full((P, Hkv, BK, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want_k, want_v = Kp.clone(), Vp.clone()
    want_k[slots // BK, :, slots % BK], want_v[slots // BK, :, slots % BK] = Ko, V
    e = err_word()
    msa.msa_qk_norm_rope(Q, K, pos, f, Q, Kp, V=V, V_out=Vp, slots=slots, q_weight=wq, k_weight=wk, interleaved=interleaved,
                         dev_err=e)
    assert torch.equal(Q, Qo) and torch.equal(Kp, want_k) and torch.equal(Vp, want_v) and int(e) == 0


def test_norm_rope_options(msa):
    """fp32 weights, no norm, no keys, a large eps, positions to 2^30, head-major strides."""
    Q, K, V, wq, wk, pos, f = rope_case(50, 6, 2, 128, 128, 3, far=1 << 30, wdtype=torch.float32)
    Qo, Ko = torch.empty_like(Q), torch.empty_like(K)
    msa.msa_qk_norm_rope(Q, K, pos, f, Qo, Ko, q_weight=wq, k_weight=wk, eps=0.5)
    check_rope(Qo, Q, wq, pos, f, False, eps=0.5)
    check_rope(Ko, K, wk, pos, f, False, eps=0.5)
    msa.msa_qk_norm_rope(Q, K, pos, f, Qo, Ko, k_weight=wk)
    check_rope(Qo, Q, None, pos, f, False)
    Qt = torch.empty(6, 50, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    msa.msa_qk_norm_rope(Q, None, pos, f, Qt, None, q_weight=wq)
    check_rope(Qt, Q, wq, pos, f, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_frequencies(msa, interleaved):
    """Frequencies of every size and sign: turns of a token from 2^-130 to 2^22, no rotation, negative ones."""
    Q, K, V, wq, wk, pos, f = rope_case(90, 2, 1, 128, 128, 8, far=1000)
    r = np.random.default_rng(3)
    v = 2.0 ** r.uniform(-126, 22.9, 64) * r.choice([-1, 1], 64)
    v[:24] = [0.0, -0.0, 2.0 ** -149, 2.0 ** -126, 1.0, -1.0, 0.5, 2.0 ** 22, 8388607.5, 2.0 ** 23, -2.0 ** 23, 2.0 ** 24 + 2, 3.14159274,
              6.28318548, -6.28318548, 1e-3, 2.0 ** -23, 2.0 ** -24, 2.0 ** -31, 2.0 ** -32, 2.0 ** -33, 2.0 ** -64, 1e5, -1e5]
    f = torch.tensor(v, dtype=torch.float32, device="cuda")
    Qo, Ko = torch.empty(90, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(90, 1, 128, dtype=torch.bfloat16, device="cuda")
    msa.msa_qk_norm_rope(Q, K, pos, f, Qo, Ko, q_weight=wq, interleaved=interleaved)
    check_rope(Qo, Q, wq, pos, f, interleaved)
    check_rope(Ko, K, None, pos, f, interleaved)


def test_norm_rope_rows_left_out(msa):
    """pos < 0 leaves a row's outputs as they were; slot < 0 stores no key; one past the pool is named."""
    N = 40
    Q, K, V, wq, wk, pos, f = rope_case(N, 4, 2, 128, 128, 9)
    pos[3::7] = -1
    slots = torch.arange(N, device="cuda") * 3
    slots[5::6] = -1
    slots[8] = 2 * BK
    Qo = torch.full_like(Q, 5.0)
    Kp, Vp = (torch.full((2, 2, BK, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    e = err_word()
    msa.msa_qk_norm_rope(Q, K, pos, f, Qo, Kp, V=V, V_out=Vp, slots=slots, q_weight=wq, k_weight=wk, dev_err=e)
    live = pos >= 0
    assert int(e) == msa.MSA_DEVERR_BAD_PAGE
    assert (Qo[~live] == 5.0).all()
    check_rope(Qo[live], Q[live], wq, pos[live], f, False)
    stored = live & (slots >= 0) & (slots < 2 * BK)
    at = slots[stored]
    assert torch.equal(Vp[at // BK, :, at % BK], V[stored])
    check_rope(Kp[at // BK, :, at % BK], K[stored], wk, pos[stored], f, False)
    rest = torch.ones(2 * BK, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (Kp.transpose(1, 2).reshape(2 * BK, 2, 128)[rest] == 9.0).all()


# ---------------------------------------------------------------------------
# 4-bit store
# ---------------------------------------------------------------------------

def store_values(N, Hkv, seed):
    """Normal rows, and rows of zeros, halfway points, tiny, huge, infinite and NaN values."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((N, Hkv, 128)) * np.exp(r.standard_normal((N, Hkv, 1)) * 3)
    if N >= 8:
        x[1] = 0.0
        x[2] = r.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -2.5], (Hkv, 128)) * 2.0 ** r.integers(-4, 5, (Hkv, 1))
        x[3] = r.standard_normal((Hkv, 128)) * 1e-4
        x[4] = r.standard_normal((Hkv, 128)) * 1e5
        x[5, :, ::19] = np.inf
        x[5, :, 7::23] = -np.inf
        x[6, :, ::37] = np.nan
        x[7] = r.integers(-127, 128, (Hkv, 128)) / 8.0
    return torch.from_numpy(x).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("N,Hkv,ks,vs", [(1, 1, 1.0, 1.0), (8, 8, 1.0, 0.25), (500, 3, 0.125, 4.0), (4100, 2, 2.0 ** -20, 2.0 ** 9)])
def test_store_and_expand_q4(msa, N, Hkv, ks, vs):
    """Codes, scales and expanded values are those of the definition, bit for bit; other slots stay."""
    P = N // BK + 3
    K, V = store_values(N, Hkv, N), store_values(N, Hkv, N + 1)
    both = torch.cat((K, V), 1)                                  # strided views, as a projection leaves them
    K, V = both[:, :Hkv], both[:, Hkv:]
    slots = torch.from_numpy(np.random.default_rng(N).permutation(P * BK)[:N]).cuda()
    slots_in = slots.clone()
    drop = torch.zeros(N, dtype=torch.bool, device="cuda")
    if N > 8:
        slots_in[9], slots_in[10] = -1, P * BK
        drop[9], drop[10] = True, True
    c = msa.q4_cache(P, Hkv, "cuda", ks, vs)
    c.K_codes.fill_(0x35), c.K_scales.fill_(0x38), c.V_codes.fill_(0x2B), c.V_scales.fill_(0x30)
    want = {n: getattr(c, n).cpu().numpy().copy() for n in ("K_codes", "K_scales", "V_codes", "V_scales")}
    e = err_word()
    msa.msa_cache_append_q4(K, V, slots_in, c, dev_err=e)
    assert int(e) == (msa.MSA_DEVERR_BAD_PAGE if N > 8 else 0)
    at = slots[~drop].cpu().numpy()
    for x, nm, gs in ((K, "K", ks), (V, "V", vs)):
        codes, scales = ref.quantise(ref.f64(x[~drop]), gs)
        zero = np.repeat(ref.E4M3[np.minimum(scales, 126)] == 0, 8, -1) | np.repeat(scales == 0x7F, 8, -1)
        want[nm + "_codes"][at // BK, :, at % BK] = np.where(zero, 0, codes)
        want[nm + "_scales"][at // BK, :, at % BK] = scales
    for nm, w in want.items():
        got = getattr(c, nm).cpu().numpy()
        if nm.endswith("codes"):                                 # -0 and +0 are the same value
            got, w = (np.where(x & 0x77 == 0, 0, x) for x in (fold(got), fold(w)))
        assert np.array_equal(got, w), nm
    pages = torch.from_numpy(np.random.default_rng(1).permutation(P)).int().cuda()
    pages_in = torch.cat((pages, torch.tensor([P, -1], dtype=torch.int32, device="cuda")))
    Ko, Vo = (torch.full((P + 2, Hkv, BK, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    e.zero_()
    msa.msa_cache_expand_q4(c, pages_in, Ko, Vo, dev_err=e)
    assert int(e) == msa.MSA_DEVERR_BAD_PAGE and (Ko[P:] == 3.0).all() and (Vo[P:] == 3.0).all()
    p = pages.cpu().numpy()
    for o, nm, gs in ((Ko, "K", ks), (Vo, "V", vs)):
        w = ref.values(getattr(c, nm + "_codes").cpu().numpy()[p], getattr(c, nm + "_scales").cpu().numpy()[p], gs)
        assert np.array_equal(ref.f64(o[:P]), w, equal_nan=True), nm


def fold(b):
    """Each half of a byte with the sign of a zero dropped."""
    lo, hi = b & 15, b >> 4
    return np.where(lo == 8, 0, lo) | (np.where(hi == 8, 0, hi) << 4)


# ---------------------------------------------------------------------------
# decode attention over the 4-bit cache
# ---------------------------------------------------------------------------

def q4_pool(msa, P, Hkv, seed, ks=1.0, vs=0.25, spread=1.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((2, P, Hkv, BK, 128)).astype(np.float32)
    x[0] *= spread * np.exp(0.5 * r.standard_normal((Hkv, 1, 128)))
    parts = []
    for y, gs in ((x[0], ks), (x[1], vs)):
        parts += ref.quantise(torch.from_numpy(y).bfloat16().double().numpy(), gs)
    return msa.Q4Cache(*[torch.from_numpy(a).cuda() for a in parts], ks, vs)


def cache_values(c):
    return (ref.values(c.K_codes.cpu().numpy(), c.K_scales.cpu().numpy(), c.k_scale),
            ref.values(c.V_codes.cpu().numpy(), c.V_scales.cpu().numpy(), c.v_scale))


def outputs(B, Hq):
    return (torch.full((B, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((B, Hq), 7.0, dtype=torch.float32, device="cuda"))


def workspace(msa, B, Hkv):
    return torch.zeros(msa.msa_attn_decode_q4_workspace_size(B, Hkv), dtype=torch.uint8, device="cuda")


def queries(B, Hq, seed, amp=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (amp * torch.randn(B, Hq, 128, generator=g, device="cuda")).bfloat16()


def check_rows(Q, O, LSE, pages_of, tokens_of, c, scale=None):
    """Every (sequence, head group) against the definition over its pages."""
    K, V = cache_values(c)
    B, Hq, _ = Q.shape
    Hkv, P = K.shape[1], K.shape[0]
    G = Hq // Hkv
    q, o, lse = ref.f64(Q), ref.f64(O), ref.f64(LSE)
    for b in range(B):
        for g in range(Hkv):
            pages, T = pages_of(b, g), tokens_of(b, g)
            keep = [(p, min(BK, T - j * BK)) for j, p in enumerate(pages) if 0 <= p < P and T > j * BK]
            Kr = np.concatenate([K[p, g, :m] for p, m in keep]) if keep else np.zeros((0, 128))
            Vr = np.concatenate([V[p, g, :m] for p, m in keep]) if keep else np.zeros((0, 128))
            h = slice(g * G, (g + 1) * G)
            ref.check_attend(o[b, h], lse[b, h], ref.attend(q[b, h], Kr, Vr, scale or ref.default_scale()))


@pytest.mark.parametrize("B,Hq,Hkv,k", [(1, 8, 8, 16), (1, 1, 1, 1), (3, 12, 2, 16), (8, 48, 8, 16), (5, 6, 2, 64), (2, 10, 2, 7),
                                        (70, 14, 2, 3), (40, 32, 4, 16), (700, 4, 2, 5), (1300, 3, 1, 2),
                                        (300, 5, 1, 64), (1, 8, 1, 64), (2, 6, 6, 33)])
def test_sparse_decode_q4(msa, B, Hq, Hkv, k):
    r = np.random.default_rng(B * 100 + k)
    P = max(2 * k, 40)
    c = q4_pool(msa, P, Hkv, B)
    rows = B * Hkv
    pt = np.stack([r.permutation(P)[:k] for _ in range(rows)])
    n = np.where(r.random(rows) < 0.3, r.integers(0, k + 1, rows), k)
    last = r.choice([1, 2, 15, 16, 17, 63, 64, 127, 128], rows)
    for i in range(rows):
        pt[i, n[i]:] = -1
    Q = queries(B, Hq, 1)
    O, LSE = outputs(B, Hq)
    ws, e = workspace(msa, B, Hkv), err_word()
    msa.msa_sparse_attn_decode_q4(Q, c, i32(pt), i32(n), i32(last), O, LSE, ws, dev_err=e)
    assert int(e) == 0
    check_rows(Q, O, LSE, lambda b, g: pt[b * Hkv + g, :n[b * Hkv + g]],
               lambda b, g: (n[b * Hkv + g] - 1) * BK + last[b * Hkv + g] if n[b * Hkv + g] else 0, c)
    # the counters are left zero, and a second call gives the same bits
    O2, L2 = outputs(B, Hq)
    msa.msa_sparse_attn_decode_q4(Q, c, i32(pt), i32(n), i32(last), O2, L2, ws, dev_err=e, scratch_zeroed=True)
    assert torch.equal(O, O2) and torch.equal(LSE, L2) and int(e) == 0
    O3, _ = outputs(B, Hq)
    msa.msa_sparse_attn_decode_q4(Q, c, i32(pt), i32(n), i32(last), O3, None, ws, softmax_scale=ref.default_scale())
    assert torch.equal(O, O3)


@pytest.mark.parametrize("B,Hq,Hkv,k", [(50, 8, 4, 16), (38, 4, 4, 16), (75, 4, 4, 4), (14, 8, 8, 4), (13, 8, 8, 3), (152, 1, 1, 9),
                                        (26, 4, 4, 64), (8, 8, 8, 32), (5, 16, 8, 64)])
def test_sparse_decode_q4_in_parts(msa, B, Hq, Hkv, k):
    """Rows in two, three and four parts, as clusters and through the workspace."""
    test_sparse_decode_q4(msa, B, Hq, Hkv, k)


DENSE = {
    "edges": ([0, 1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000], 12, 2),
    "one": ([1], 1, 1),
    "long_row": ([40000], 6, 1),
    "gqa8": ([9000, 0, 640, 3], 16, 2),
    "gqa1": ([300, 4100, 777], 3, 3),
    "many": ([(37 * i) % 700 for i in range(150)], 8, 4),
    "b600": ([(53 * i) % 401 for i in range(600)], 3, 1),
    "b1024": ([(i % 3) * ((17 * i) % 260) for i in range(1024)], 2, 1),
    "one_long_of_many": ([3] * 200 + [30000] + [0] * 50 + [129] * 100, 2, 1),
    "all_empty": ([0] * 40, 6, 2),
    "two_long": ([50000, 21], 4, 2),
}


@pytest.mark.parametrize("name", DENSE)
def test_dense_decode_q4(msa, name):
    L, Hq, Hkv = DENSE[name]
    B = len(L)
    per = [-(-x // BK) for x in L]
    P, mp = sum(per) + 2, max(max(per), 1) + 1
    c = q4_pool(msa, P, Hkv, 3)
    ids, at = np.random.default_rng(2).permutation(P), 0
    pt = np.full((B, mp), -1)
    for b in range(B):
        pt[b, :per[b]] = ids[at:at + per[b]]
        at += per[b]
    Q = queries(B, Hq, 2)
    O, LSE = outputs(B, Hq)
    ws, e = workspace(msa, B, Hkv), err_word()
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O, LSE, ws, dev_err=e)
    assert int(e) == 0
    check_rows(Q, O, LSE, lambda b, g: pt[b, :per[b]], lambda b, g: L[b], c)
    O2, L2 = outputs(B, Hq)
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O2, L2, ws, scratch_zeroed=True)
    assert torch.equal(O, O2) and torch.equal(LSE, L2)


@pytest.mark.parametrize("L,Hq,Hkv", [([150 * BK], 2, 1), ([149 * BK + 5] * 2, 3, 1), ([190000] + [30 * BK] * 49, 2, 2), ([60 * BK + 1], 5, 1),
                                      ([120000] + [7] * 400, 1, 1)])
def test_dense_decode_q4_many_parts(msa, L, Hq, Hkv):
    """Rows in so many parts that they are joined in groups; pages shared, so that the pool is small."""
    r, P, B = np.random.default_rng(7), 50, len(L)
    per = [-(-x // BK) for x in L]
    pt = r.integers(0, P, (B, max(per) + 3))
    c, Q = q4_pool(msa, P, Hkv, 5), queries(B, Hq, 3)
    O, LSE = outputs(B, Hq)
    ws = workspace(msa, B, Hkv)
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O, LSE, ws)
    check_rows(Q, O, LSE, lambda b, g: pt[b, :per[b]], lambda b, g: L[b], c)
    for _ in range(3):
        O2, L2 = outputs(B, Hq)
        msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O2, L2, ws, scratch_zeroed=True)
        assert torch.equal(O, O2) and torch.equal(LSE, L2)


@pytest.mark.parametrize("L,Hq,Hkv", [([437 + 35 * i for i in range(40)], 2, 1), ([1 + 26 * i for i in range(20)], 8, 8),
                                      ([129] * 152, 1, 1), ([129 + i for i in range(153)], 1, 1), ([0, 300, 0, 1] * 19, 4, 4),
                                      ([640] * 77, 4, 4), ([1500] * 30 + [0], 5, 5), ([20000, 1, 1, 0], 2, 1)])
def test_dense_decode_q4_whole_parts(msa, L, Hq, Hkv):
    """Around the sizes from which CTAs take whole parts of rows, and four warps instead of eight."""
    test_dense_decode_q4_many_parts(msa, L, Hq, Hkv)


@pytest.mark.parametrize("amp,spread", [(40.0, 4.0), (1e-3, 1e-2), (2.0 ** 100, 2.0 ** -3), (0.0, 1.0)])
def test_decode_q4_score_ranges(msa, amp, spread):
    """Scores that concentrate on one token, that are all alike, queries far outside fp16's range, and zeros."""
    c = q4_pool(msa, 12, 2, 8, spread=spread)
    L = [700, 333]
    pt = np.arange(12).reshape(2, 6)
    Q = queries(2, 12, 4, amp)
    O, LSE = outputs(2, 12)
    scale = ref.default_scale() if amp < 1e6 else 2.0 ** -97
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O, LSE, workspace(msa, 2, 2), softmax_scale=scale)
    check_rows(Q, O, LSE, lambda b, g: pt[b], lambda b, g: L[b], c, scale)


def test_decode_q4_rising_scores(msa):
    """Keys that grow along the row: the running maximum is raised again and again."""
    c = q4_pool(msa, 20, 1, 9)
    Kv = ref.f64(queries(20 * BK, 1, 5)).reshape(20, 1, BK, 128) * 0.05
    Kv += np.linspace(0, 3, 20 * BK).reshape(20, 1, BK, 1)
    codes, scales = ref.quantise(torch.from_numpy(Kv).bfloat16().double().numpy(), 1.0)
    c = c._replace(K_codes=torch.from_numpy(codes).cuda(), K_scales=torch.from_numpy(scales).cuda())
    Q = (torch.ones(1, 4, 128, device="cuda") * torch.tensor([1.0, -1.0, 0.3, 3.0], device="cuda")[:, None]).bfloat16()
    pt = np.arange(20)[None]
    O, LSE = outputs(1, 4)
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32([2500]), O, LSE, workspace(msa, 1, 1))
    check_rows(Q, O, LSE, lambda b, g: pt[0], lambda b, g: 2500, c)


def test_decode_q4_unused_slots_and_pages(msa):
    """Slots past the last token and pages that no row lists may hold anything, NaN scales too; a NaN in a live
    token reaches exactly its own group's heads."""
    L, Hq, Hkv = [131, 250], 6, 2
    c = q4_pool(msa, 6, Hkv, 12)
    pt = np.array([[4, 1], [0, 3]])
    clean = outputs(2, Hq)
    Q, ws = queries(2, Hq, 6), workspace(msa, 2, Hkv)
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), *clean, ws)
    for t in (c.K_scales, c.V_scales):
        t[[2, 5]] = 0x7F
        t[1, :, 3:] = 0x7F
        t[3, :, 250 - BK:] = 0x7F
    O, LSE = outputs(2, Hq)
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O, LSE, ws)
    assert torch.equal(O, clean[0]) and torch.equal(LSE, clean[1])
    rows_pt = np.repeat(pt, Hkv, 0)
    msa.msa_sparse_attn_decode_q4(Q, c, i32(rows_pt), i32([2] * 4), i32([3, 3, 122, 122]), O, LSE, ws)
    check_rows(Q, O, LSE, lambda b, g: pt[b], lambda b, g: L[b], c)
    c.V_scales[0, 1, 77, 2] = 0x7F
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O, LSE, ws)
    assert torch.equal(O[0], clean[0][0]) and torch.equal(O[1, :3], clean[0][1, :3])
    assert torch.isnan(O[1, 3:, 32:48]).all() and not torch.isnan(O[1, 3:, :32]).any()
    c.K_scales[0, 0, 5, 0] = 0x7F
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O, LSE, ws)
    assert torch.isnan(O[1, :3]).all() and torch.isnan(LSE[1, :3]).all() and torch.equal(O[0], clean[0][0])


def test_decode_q4_bad_pages_and_lengths(msa):
    L, Hq, Hkv = [500, 300, -3, 2000], 4, 2
    c = q4_pool(msa, 9, Hkv, 13)
    pt = np.array([[0, 9, 2, 3], [4, 5, -2, -1], [6, 7, 8, 1], [6, 7, 8, 1]])
    Q, ws, e = queries(4, Hq, 7), workspace(msa, 4, Hkv), err_word()
    O, LSE = outputs(4, Hq)
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O, LSE, ws, dev_err=e)
    assert int(e) == msa.MSA_DEVERR_BAD_PAGE | msa.MSA_DEVERR_BAD_LEN
    check_rows(Q, O, LSE, lambda b, g: pt[b], lambda b, g: L[b] if b < 2 else 0, c)
    # sparse: counts and last lengths outside their ranges are taken within them
    n, last = [9, 3, 4, -1, 2, 2, 1, 1], [500, 128, 0, 5, -4, 7, 128, 128]
    rows_pt = np.repeat(pt, Hkv, 0)
    e.zero_()
    msa.msa_sparse_attn_decode_q4(Q, c, i32(rows_pt), i32(n), i32(last), O, LSE, ws, dev_err=e)
    assert int(e) == msa.MSA_DEVERR_BAD_PAGE
    T = [0 if a <= 0 else (min(a, 4) - 1) * BK + min(max(b, 0), BK) for a, b in zip(n, last)]
    check_rows(Q, O, LSE, lambda b, g: pt[b], lambda b, g: T[b * Hkv + g], c)


def test_q4_strided_pools_and_queries(msa):
    """One layer's K and V of a pool that interleaves layers and sides, and Q as a slice of a projection: what dense
    tensors give."""
    P, Hkv, Hq, L = 12, 2, 12, [700, 333]
    c = q4_pool(msa, P, Hkv, 15)
    codes = torch.full((P, 3, 2, Hkv, BK, 64), 0xFF, dtype=torch.uint8, device="cuda")
    scales = torch.full((P, 3, 2, Hkv, BK, 8), 0x7F, dtype=torch.uint8, device="cuda")
    s = msa.Q4Cache(codes[:, 1, 0], scales[:, 1, 0], codes[:, 1, 1], scales[:, 1, 1], c.k_scale, c.v_scale)
    every = torch.arange(P, dtype=torch.int32, device="cuda")
    for a, b in zip(s[:4], c[:4]):
        a.copy_(b)
    pt = np.random.default_rng(3).permutation(P).reshape(2, 6)
    wide = queries(2, Hq + 5, 16)
    Q, ws = wide[:, 3:3 + Hq], workspace(msa, 2, Hkv)
    want, got = outputs(2, Hq), outputs(2, Hq)
    msa.msa_dense_attn_decode_q4(Q.contiguous(), c, i32(pt), i32(L), *want, ws)
    msa.msa_dense_attn_decode_q4(Q, s, i32(pt), i32(L), *got, ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    K = queries(40, Hkv, 17, 1.0)
    slots = torch.randperm(P * BK, device="cuda")[:40]
    out = [[torch.empty(P, Hkv, BK, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    for x, o in ((c, out[0]), (s, out[1])):
        msa.msa_cache_append_q4(K, K, slots, x)
        msa.msa_cache_expand_q4(x, every, *o)
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert (codes[:, [0, 2]] == 0xFF).all() and (scales[:, [0, 2]] == 0x7F).all()


def test_decode_q4_on_two_streams_at_once(msa):
    """Two attentions in flight with workspaces of their own, many times over: the bits of calls one by one."""
    c = q4_pool(msa, 30, 2, 18)
    pt, L = i32(np.arange(30).reshape(3, 10)), i32([1280, 900, 77])
    Qs, ws, want = [queries(3, 12, 20 + i) for i in range(2)], [workspace(msa, 3, 2) for _ in range(2)], []
    for i in range(2):
        want.append(outputs(3, 12))
        msa.msa_dense_attn_decode_q4(Qs[i], c, pt, L, *want[i], ws[i])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[outputs(3, 12) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for r in range(20):
        for i in range(2):
            msa.msa_dense_attn_decode_q4(Qs[i], c, pt, L, *got[i][r], ws[i], stream=streams[i], scratch_zeroed=True)
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o[0], want[i][0]) and torch.equal(o[1], want[i][1])


def test_decode_q4_workspace_of_several_shapes(msa):
    """One zero-filled workspace of the largest size, calls of both kinds and several shapes in turn."""
    c, ws = q4_pool(msa, 60, 4, 21), workspace(msa, 64, 4)
    calls = []
    for B, seed in ((3, 1), (1, 2), (6, 3), (64, 4)):
        Q = queries(B, 16, 30 + seed)
        pt = i32(np.arange(B * 16).reshape(B, 16) % 60)
        L = i32(np.full(B, 2000) - np.arange(B))
        rows = i32(np.arange(B * 4 * 16).reshape(B * 4, 16) % 60)
        n, last = i32(np.full(B * 4, 16)), i32(np.full(B * 4, 100))
        calls.append((msa.msa_dense_attn_decode_q4, (Q, c, pt, L), outputs(B, 16), workspace(msa, B, 4)))
        calls.append((msa.msa_sparse_attn_decode_q4, (Q, c, rows, n, last), outputs(B, 16), workspace(msa, B, 4)))
    for f, args, want, own in calls:
        f(*args, *want, own)
    for order in (calls, calls[::-1]):
        for f, args, want, _ in order:
            got = outputs(*want[1].shape)
            f(*args, *got, ws, scratch_zeroed=True)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_serving_calls_without_rows(msa):
    c, e = q4_pool(msa, 2, 2, 1), torch.empty
    bf, i64, dev = torch.bfloat16, torch.int64, "cuda"
    none, K = i32([]), e(0, 2, 128, dtype=bf, device=dev)
    msa.msa_qk_norm_rope(e(0, 4, 128, dtype=bf, device=dev), K, none, None, e(0, 4, 128, dtype=bf, device=dev), K)
    msa.msa_cache_append_q4(K, K, e(0, dtype=i64, device=dev), c)
    blocks = e(0, 2, 128, 128, dtype=bf, device=dev)
    msa.msa_cache_expand_q4(c, none, blocks, blocks)
    Q, table, ws = e(0, 4, 128, dtype=bf, device=dev), e(0, 3, dtype=torch.int32, device=dev), workspace(msa, 1, 2)
    msa.msa_sparse_attn_decode_q4(Q, c, table, none, none, Q, None, ws)
    msa.msa_dense_attn_decode_q4(Q, c, table, none, Q, None, ws)
    torch.cuda.synchronize()


def test_decode_q4_far_pages(msa):
    """A pool whose last page lies past 2^32 bytes."""
    Hkv, P = 8, 68000                                            # 8192 code bytes a block: 4.46e9
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("needs 16 GB")
    c = msa.q4_cache(P, Hkv, "cuda")
    small = q4_pool(msa, 3, Hkv, 14, vs=1.0)
    for big, s in zip(c[:4], small[:4]):
        big[P - 3:] = s
    pt, L = np.array([[P - 1, P - 3, P - 2]]), [300]
    Q, ws = queries(1, 48, 8), workspace(msa, 1, Hkv)
    O, LSE = outputs(1, 48)
    msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O, LSE, ws)
    check_rows(Q, O, LSE, lambda b, g: pt[0] - (P - 3), lambda b, g: 300, small)
    K = queries(2, Hkv, 9, 1.0)
    slots = torch.tensor([P * BK - 1, (P - 1) * BK], device="cuda")
    msa.msa_cache_append_q4(K, K, slots, c)
    Ko, Vo = (torch.empty(1, Hkv, BK, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    msa.msa_cache_expand_q4(c, i32([P - 1]), Ko, Vo)
    want = ref.values(*ref.quantise(ref.f64(K), 1.0), 1.0)
    assert np.array_equal(ref.f64(Ko[0, :, 127]), want[0]) and np.array_equal(ref.f64(Vo[0, :, 0]), want[1])


# ---------------------------------------------------------------------------
# refusals, streams
# ---------------------------------------------------------------------------

def test_wrappers_refuse_on_the_gpu(msa):
    from test_serving_abi import wrapper_refusals
    for i, refused in enumerate(wrapper_refusals("cuda")):
        with pytest.raises(ValueError):
            refused()
            raise AssertionError(f"call {i} was accepted")
    L, pt = i32([3]), i32([[0]])
    with pytest.raises(msa.MSAError):                            # a workspace that is too small: the entry point's refusal
        msa.msa_dense_attn_decode_q4(queries(1, 2, 0), msa.q4_cache(3, 2, "cuda"), pt, L, *outputs(1, 2), err_word())


def test_stream_arguments(msa):
    """A torch stream, its raw pointer and the current stream: work goes where it is sent."""
    c = PLANS["edges"]()
    want = ref.plan(*c)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, None):
        t = [i32(x) for x in (c[0], c[1], c[2], c[3], [c[4]])]
        o = msa.plan_buffers(len(c[0]), c[5], "cuda")
        torch.cuda.synchronize()
        msa.msa_plan_step(*t, *o.values(), num_pages=c[6], stream=stream)
        (torch.cuda.current_stream() if stream is None else side).synchronize()
        assert np.array_equal(o["tok_slot"].cpu(), want["tok_slot"]) and np.array_equal(o["cu"].cpu(), want["cu"])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def serving_state(msa, B, Hq, Hkv, N, mp, pool, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"seq_len": torch.zeros(B, dtype=torch.int32, device="cuda"), "seq_pt": torch.full((B, mp), -1, dtype=torch.int32, device="cuda"),
         "free": torch.randperm(pool, generator=g, device="cuda").int(), "count": i32([pool]),
         "new": torch.zeros(B, dtype=torch.int32, device="cuda"),
         "qkv": torch.zeros(N, Hq + 2 * Hkv, 128, dtype=torch.bfloat16, device="cuda"),
         "K": torch.zeros(N, Hkv, 128, dtype=torch.bfloat16, device="cuda"),
         "Q": torch.zeros(N, Hq, 128, dtype=torch.bfloat16, device="cuda"),
         "w": [(1 + 0.1 * torch.randn(128, generator=g, device="cuda")).bfloat16() for _ in range(2)],
         "f": (1e4 ** (-torch.arange(0, 128, 2, device="cuda").double() / 128)).float(),
         "plan": msa.plan_buffers(B, N, "cuda"), "cache": msa.q4_cache(pool, Hkv, "cuda", 1.0, 0.5), "err": err_word(),
         "O": torch.zeros(B, Hq, 128, dtype=torch.bfloat16, device="cuda"), "LSE": torch.zeros(B, Hq, device="cuda"),
         "Qlast": torch.zeros(B, Hq, 128, dtype=torch.bfloat16, device="cuda"), "ws": workspace(msa, B, Hkv)}
    return s


def serving_step(msa, s, Hq, Hkv):
    """Slots, norm with rotation, 4-bit store and attention of each request's newest token."""
    p = s["plan"]
    msa.msa_plan_step(s["seq_len"], s["new"], s["seq_pt"], s["free"], s["count"], s["seq_len"], s["count"], p["cu"],
                      p["tok_slot"], p["tok_pos"], p["tok_seq"], num_pages=s["free"].shape[0], dev_err=s["err"])
    x = s["qkv"]
    msa.msa_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], p["tok_pos"], s["f"], s["Q"], s["K"], q_weight=s["w"][0],
                         k_weight=s["w"][1], dev_err=s["err"])
    msa.msa_cache_append_q4(s["K"], x[:, Hq + Hkv:], p["tok_slot"], s["cache"], dev_err=s["err"])
    s["Qlast"].copy_(s["Q"][(p["cu"][1:].long() - 1).clamp(min=0)])
    msa.msa_dense_attn_decode_q4(s["Qlast"], s["cache"], s["seq_pt"], s["seq_len"], s["O"], s["LSE"], s["ws"],
                                 dev_err=s["err"], scratch_zeroed=True)


@pytest.mark.parametrize("captured", [False, True])
def test_serving_run(msa, captured):
    """Prompts, then single tokens, then an ended request's pages reused; eager on a side stream, or one captured graph
    replayed: every step against the definitions over the tokens fed so far."""
    B, Hq, Hkv, N, mp, pool = 5, 12, 2, 700, 8, 24
    s = serving_state(msa, B, Hq, Hkv, N, mp, pool)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    fed_k, fed_v = [[] for _ in range(B)], [[] for _ in range(B)]
    graph = None
    r = np.random.default_rng(4)
    with torch.cuda.stream(stream):
        if captured:
            serving_step(msa, s, Hq, Hkv)                        # no request brings a token: nothing changes
            graph = torch.cuda.CUDAGraph()
            stream.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                serving_step(msa, s, Hq, Hkv)
        for step, new in enumerate([[200, 1, 130, 0, 128], [1, 1, 1, 300, 1], [1, 1, 0, 1, 127], [2, 1, 400, 1, 1]]):
            if step == 3:                                        # request 2 ends; its row takes a new prompt
                done = i32([0, 0, 1, 0, 0])
                msa.msa_release_pages(s["seq_len"], done, s["seq_pt"], s["free"], s["count"], s["seq_len"], s["count"])
                fed_k[2], fed_v[2] = [], []
            s["new"].copy_(i32(new))
            x = torch.from_numpy(r.standard_normal(s["qkv"].shape)).bfloat16()
            s["qkv"].copy_(x)
            graph.replay() if captured else serving_step(msa, s, Hq, Hkv)
            stream.synchronize()
            assert int(s["err"]) == 0
            row, K = 0, s["K"].cpu()
            for b, n in enumerate(new):
                for i in range(row, row + n):
                    fed_k[b].append(ref.f64(K[i])), fed_v[b].append(ref.f64(x[i, Hq + Hkv:]))
                row += n
            check_rope(s["K"][:row], x[:row, Hq:Hq + Hkv], s["w"][1], s["plan"]["tok_pos"][:row], s["f"], False)
            assert s["seq_len"].tolist() == [len(v) for v in fed_k]
            for b in range(B):
                T = len(fed_k[b])
                kv = [ref.values(*ref.quantise(np.array(v).reshape(T, Hkv, 128), gs), gs) for v, gs in ((fed_k[b], 1.0), (fed_v[b], 0.5))]
                for g in range(Hkv):
                    h = slice(g * 6, g * 6 + 6)
                    ref.check_attend(ref.f64(s["O"][b, h]), ref.f64(s["LSE"][b, h]), ref.attend(
                        ref.f64(s["Qlast"][b, h]), kv[0][:, g], kv[1][:, g], ref.default_scale()))


def test_decode_step_q4_follows_the_selection(msa):
    """The MSA step over the 4-bit cache: the same selection as over bf16 pools, and the attention of the cached values."""
    from workloads import DecodeWorkload, MSAShape, decode_inputs
    wl = DecodeWorkload("q4_step", lengths=(1, 700, 5000, 2050), shape=MSAShape(Hq=12, Hkv=2, k=4), seed=61)
    inp = decode_inputs(wl, device="cuda")
    P, Hkv = inp["K_pool"].shape[:2]
    c = msa.q4_cache(P, Hkv, "cuda", 2.0 ** -6, 2.0 ** -6)
    rows = lambda x: x.transpose(1, 2).reshape(P * BK, Hkv, 128)  # noqa: E731
    msa.msa_cache_append_q4(rows(inp["K_pool"]), rows(inp["V_pool"]), torch.arange(P * BK, device="cuda"), c)
    a, b = msa.decode_step(inp, 4), msa.decode_step_q4(inp, c, 4)
    assert int(a["dev_err"]) == 0 and int(b["dev_err"]) == 0
    for nm in ("sel", "count", "pt", "n", "last_len"):
        assert torch.equal(a[nm], b[nm]), nm
    pt, n, last = (b[x].cpu().numpy() for x in ("pt", "n", "last_len"))
    check_rows(inp["Q"], b["O"], b["LSE"], lambda i, g: pt[i * Hkv + g, :n[i * Hkv + g]],
               lambda i, g: (n[i * Hkv + g] - 1) * BK + last[i * Hkv + g], c)
    # the 4-bit pages expanded give the bf16 step the same values
    Ko, Vo = torch.empty_like(inp["K_pool"]), torch.empty_like(inp["V_pool"])
    msa.msa_cache_expand_q4(c, torch.arange(P, dtype=torch.int32, device="cuda"), Ko, Vo)
    d = msa.decode_step(dict(inp, K_pool=Ko, V_pool=Vo), 4)
    assert torch.allclose(d["O"].float(), b["O"].float(), atol=2e-3, rtol=2 ** -6) and math.isfinite(float(d["LSE"].sum()))
