"""Cases of the step around paged attention over a 4-bit cache: page tables and
token slots from request lengths, per-head norm with position rotation, the
4-bit store, and decode attention that reads it.

Head layout and lengths are those of the framework's workloads (48 query heads
over 8 KV heads of 128, 128-token pages, 16 selected pages, 60,001 and 1,048,576
cached tokens).  ``own`` chooses between the plain form (elementary torch
operations in 32 bits) and the framework's calls.
"""
import math

import torch

own = False

BK = 128                      # tokens per page
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # magnitudes of a 4-bit float (1 sign, 2 exponent, 1 mantissa bit)


def listed():
    return [
        # one token for each of 8 running requests: the table update before every decode step
        dict(name="tables_b8", op="tables", B=8, fresh=0, done=0, new_lo=1, new_hi=1, ctx_lo=60001, ctx_hi=60001,
             max_pages=512, pad=0),
        # a scheduler step of a busy server: requests that end, requests that start with a prompt, the rest go on by one
        # token; the token rows are padded to the size of a captured graph
        dict(name="tables_turnover_b64", op="tables", B=64, fresh=8, done=6, new_lo=1000, new_hi=9000, ctx_lo=4096,
             ctx_hi=524288, max_pages=4224, pad=311),
        # many short requests, prompts admitted together
        dict(name="tables_turnover_b1024", op="tables", B=1024, fresh=200, done=170, new_lo=16, new_hi=1500, ctx_lo=1,
             ctx_hi=32768, max_pages=300, pad=0),
        # one decode step of 8 sequences
        dict(name="rope_b8", op="rope", N=8, Hq=48, Hkv=8, D=128, rot=128, interleaved=False, values=True, far=1048576),
        # index queries (4 heads in each of 8 groups) and index keys of a chunk, half of each head rotated in pairs
        dict(name="rope_index_n4097", op="rope", N=4097, Hq=32, Hkv=8, D=64, rot=32, interleaved=True, values=False,
             far=131072),
        # a long prefill
        dict(name="rope_n65536", op="rope", N=65536, Hq=48, Hkv=8, D=128, rot=128, interleaved=False, values=True,
             far=65536),
        # 8 decoded tokens into their pages, and these pages read back
        dict(name="store_b8", op="store", B=8, T=1, Hkv=8),
        # a prefill chunk of 8,192 tokens stored, and its pages expanded for the chunk's attention
        dict(name="store_chunk_t8192", op="store", B=1, T=8192, Hkv=8),
        # decode over the selected pages, 8 sequences
        dict(name="sparse_b8", op="sparse", B=8, Hq=48, Hkv=8, k=16, short=False),
        # a large batch, with sequences that have fewer pages than are selected and one padding row
        dict(name="sparse_b192", op="sparse", B=192, Hq=48, Hkv=8, k=16, short=True),
        # decode over every cached token
        dict(name="dense_b8_l60001", op="dense", B=8, Hq=48, Hkv=8, lo=60001, hi=60001),
        dict(name="dense_b1_l1048576", op="dense", B=1, Hq=48, Hkv=8, lo=1048576, hi=1048576),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "store", "sparse", "dense", "dense"])
    if op == "tables":
        B = _log(rng, 1, 1024)
        max_pages = _log(rng, 8, 4096 if B <= 64 else 512)
        new_hi = _log(rng, 1, min(9000, max_pages * BK // 2, max(1, 262144 // B)))
        fresh = rng.randint(0, B // 2)
        return dict(op=op, B=B, fresh=fresh, done=rng.randint(0, B - fresh), new_lo=_log(rng, 1, new_hi), new_hi=new_hi,
                    ctx_lo=1, ctx_hi=_log(rng, 1, max_pages * BK // 2), max_pages=max_pages, pad=rng.choice([0, 1, 77, 1000]))
    if op == "rope":
        D = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, N=_log(rng, 1, 32768), Hq=Hkv * rng.choice([1, 3, 4, 6, 8]), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, D // 4]), interleaved=rng.random() < 0.4, values=rng.random() < 0.7,
                    far=_log(rng, 1000, 1048576))
    if op == "store":
        T = _log(rng, 1, 8192)
        return dict(op=op, B=_log(rng, 1, max(1, min(128, 8192 // T))), T=T, Hkv=rng.choice([1, 2, 4, 8]))
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op == "sparse":
        return dict(op=op, B=_log(rng, 1, 192), Hq=Hq, Hkv=Hkv, k=rng.choice([1, 4, 8, 16, 16, 24, 32]), short=rng.random() < 0.5)
    B = _log(rng, 1, 64)
    hi = _log(rng, 1, max(1, 1000000 // B))
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, lo=_log(rng, 1, hi), hi=hi)


# ---------------------------------------------------------------------------
# sizes that follow from a case alone
# ---------------------------------------------------------------------------

def _spread(n, lo, hi, turn):
    """n lengths over [lo, hi], evenly on a logarithmic scale, in an order of their own."""
    if lo >= hi:
        return [lo] * n
    return [max(lo, min(hi, int(lo * (hi / lo) ** ((((i * 37 + turn) % n) + 0.5) / n)))) for i in range(n)]


def _table_lengths(c):
    """(cached tokens, new tokens, done) of each request: `done` ones end, `fresh` ones start, the others go on by one token."""
    B = c["B"]
    L, n = _spread(B, c["ctx_lo"], c["ctx_hi"], 5), [1] * B
    done = [False] * B
    prompts = _spread(max(1, c["fresh"]), c["new_lo"], c["new_hi"], 3)
    for i in range(c["fresh"]):
        b = i * B // max(1, c["fresh"])
        L[b], n[b] = 0, prompts[i]
    left = c["done"]
    for b in range(B - 1, -1, -1):
        if left and L[b] > 0:
            done[b], n[b], left = True, 0, left - 1
    return L, n, done


def _dense_lengths(c):
    return _spread(c["B"], c["lo"], c["hi"], 1)


def _sparse_counts(c):
    """(selected pages, valid tokens of the last one) of each sequence; a padding sequence has none."""
    n, last = [], []
    for b in range(c["B"]):
        short = c["short"] and b % 5 == 3
        n.append(1 + (b * 7) % c["k"] if short else c["k"])
        last.append(1 + (b * 53 + 60000) % BK)
    if c["short"] and c["B"] > 1:
        n[-1], last[-1] = 0, 0
    return n, last


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _fill_cache(g, pages, Hkv):
    """A 4-bit cache of normal keys (some channels larger, as trained keys have) and values."""
    chan = torch.exp(0.4 * _normal(g, Hkv, 1, 128))
    c = {"k_scale": 1.0, "v_scale": 0.25}
    for side, gs in (("K", 1.0), ("V", 0.25)):
        codes = torch.empty(pages, Hkv, BK, 64, dtype=torch.uint8, device="cuda")
        scales = torch.empty(pages, Hkv, BK, 8, dtype=torch.uint8, device="cuda")
        for p in range(0, pages, 1024):
            x = _normal(g, min(1024, pages - p), Hkv, BK, 128)
            codes[p:p + 1024], scales[p:p + 1024] = _quantise((x * chan if side == "K" else x).bfloat16(), gs)
        c[side + "_codes"], c[side + "_scales"] = codes, scales
    return c


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "tables":
        L, n, done = _table_lengths(case)
        B, mp = case["B"], case["max_pages"]
        need = sum((a + b + BK - 1) // BK for a, b in zip(L, n))
        pool = need + B + 16
        ids = torch.randperm(pool, generator=g, device="cuda").int()
        have = _ints([(a + BK - 1) // BK for a in L])
        at = torch.cumsum(have, 0) - have
        j = torch.arange(mp, device="cuda")
        seq_pt = torch.where(j < have[:, None], ids[(at[:, None] + j).clamp(max=pool - 1)], torch.full_like(ids[:1], -1))
        used = int(have.sum())
        free = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        free[:pool - used] = ids[used:]
        N = sum(n) + case["pad"]
        s = {"seq_len": _ints(L), "new_len": _ints(n), "done": _ints([int(d) for d in done]), "seq_pt": seq_pt,
             "free_pages": free, "free_count": _ints([pool - used]), "num_pages": pool, "any_done": any(done), "N": N}
        s["out"] = {"mid_len": torch.empty(B, dtype=torch.int32, device="cuda"), "mid_free": _ints([0]),
                    "seq_len": torch.empty(B, dtype=torch.int32, device="cuda"), "free_count": _ints([0]),
                    "cu": torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                    "slot": torch.empty(N, dtype=torch.int64, device="cuda"),
                    "pos": torch.empty(N, dtype=torch.int32, device="cuda"),
                    "seq": torch.empty(N, dtype=torch.int32, device="cuda"), "err": _ints([0])}
    elif op == "rope":
        N, Hq, Hkv, D = case["N"], case["Hq"], case["Hkv"], case["D"]
        heads = Hq + (2 if case["values"] else 1) * Hkv
        qkv = (1.3 * _normal(g, N, heads, D)).bfloat16()       # the projection's output: Q, K (and V) side by side
        P = (N + BK - 1) // BK + 1
        slots = torch.randperm(P, generator=g, device="cuda")[torch.arange(N, device="cuda") // BK] * BK \
            + torch.arange(N, device="cuda") % BK
        base = 5000000.0
        s = {"Q": qkv[:, :Hq], "K": qkv[:, Hq:Hq + Hkv], "V": qkv[:, Hq + Hkv:] if case["values"] else None,
             "q_weight": (1 + 0.2 * _normal(g, D)).bfloat16(), "k_weight": (1 + 0.2 * _normal(g, D)).bfloat16(),
             "pos": (max(0, case["far"] - N) + torch.arange(N, device="cuda")).int(),
             "inv_freq": (base ** (-torch.arange(0, case["rot"], 2, device="cuda").double() / case["rot"])).float(),
             "slots": slots, "rot": case["rot"], "interleaved": case["interleaved"], "eps": 1e-6,
             "Q_out": torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda"),
             "K_pool": torch.zeros(P, Hkv, BK, D, dtype=torch.bfloat16, device="cuda"),
             "V_pool": torch.zeros(P, Hkv, BK, D, dtype=torch.bfloat16, device="cuda") if case["values"] else None,
             "err": _ints([0])}
    elif op == "store":
        B, T, Hkv = case["B"], case["T"], case["Hkv"]
        start = [(b * 29 + 1) % BK for b in range(B)]          # tokens already in each sequence's first page
        per = [(a + T + BK - 1) // BK for a in start]
        pages = torch.randperm(sum(per), generator=g, device="cuda").int()
        first = [sum(per[:b]) for b in range(B)]
        at = torch.cat([torch.arange(a, a + T) + f * BK for a, f in zip(start, first)]).cuda()
        chan = torch.exp(0.4 * _normal(g, Hkv, 128))
        s = _fill_cache(g, sum(per), Hkv)
        s |= {"K": (_normal(g, B * T, Hkv, 128) * chan).bfloat16(), "V": _normal(g, B * T, Hkv, 128).bfloat16(),
              "slots": pages[at // BK].long() * BK + at % BK, "pages": pages, "err": _ints([0])}
        for x in ("K", "V"):
            s[x + "_out"] = torch.empty(sum(per), Hkv, BK, 128, dtype=torch.bfloat16, device="cuda")
    else:
        B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
        s = {"Q": (1.5 * _normal(g, B, Hq, 128)).bfloat16(), "scale": 1 / math.sqrt(128.0), "err": _ints([0])}
        if op == "sparse":
            k = case["k"]
            n, last = _sparse_counts(case)
            pool = max(B * k * 2, 64)                           # a cache that holds more than the selected pages
            pick = torch.rand(B * Hkv, pool // B, generator=g, device="cuda").argsort(1)[:, :k] \
                + (torch.arange(B * Hkv, device="cuda") // Hkv * (pool // B))[:, None]
            live = torch.arange(k, device="cuda") < _ints(n).repeat_interleave(Hkv)[:, None]
            s |= {"pt": torch.where(live, pick, torch.full_like(pick, -1)).int(), "n": _ints(n).repeat_interleave(Hkv),
                  "last_len": _ints(last).repeat_interleave(Hkv), "k": k}
        else:
            L = _dense_lengths(case)
            per = [(a + BK - 1) // BK for a in L]
            pool = sum(per)
            ids = torch.randperm(pool, generator=g, device="cuda").int()
            seq_pt = torch.full((B, max(per)), -1, dtype=torch.int32, device="cuda")
            for b in range(B):
                seq_pt[b, :per[b]] = ids[sum(per[:b]):sum(per[:b + 1])]
            s |= {"seq_pt": seq_pt, "seq_len": _ints(L),
                  # which (sequence, block) each cached page is, as the program's scheduler knows it
                  "unit_seq": torch.repeat_interleave(torch.arange(B), torch.tensor(per)).cuda(),
                  "unit_block": torch.cat([torch.arange(p) for p in per]).cuda()}
        s |= _fill_cache(g, pool, Hkv)
        s["O"] = torch.empty(B, Hq, 128, dtype=torch.bfloat16, device="cuda")
        s["LSE"] = torch.empty(B, Hq, dtype=torch.float32, device="cuda")
        # scratch, as a program keeps it: zero-filled, and large enough for any split of the work
        s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    s["op"] = op
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _quantise(x, gs):
    """codes [.., D/2] (element 2i in the low half of byte i) and group scales [.., D/16] of x [.., D]."""
    x = x.float()
    groups = x.reshape(*x.shape[:-1], -1, 16)
    scale = (groups.abs().amax(-1) / (6.0 * gs)).clamp(max=448.0).to(torch.float8_e4m3fn)
    q = groups / (scale.float() * gs)[..., None]
    a = torch.where(scale.float()[..., None] == 0, torch.zeros_like(q), q).abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5).int())
    code = (code + 8 * (groups < 0).int()).reshape(x.shape)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), scale.view(torch.uint8)


def _values(codes, scales, gs):
    """What a 4-bit block stands for, in 32 bits."""
    table = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).long()].reshape(*codes.shape[:-1], -1, 16)
    return (v * (scales.view(torch.float8_e4m3fn).float() * gs)[..., None]).flatten(-2)


def _plain_tables(s):
    L, n, seq_pt, stack, count = s["seq_len"], s["new_len"], s["seq_pt"], s["free_pages"], s["free_count"]
    j = torch.arange(seq_pt.shape[1], device=L.device)
    if s["any_done"]:                                           # the pages of ended requests go back on the stack
        gone = torch.where(s["done"] != 0, (L + BK - 1) // BK, 0)
        at = count + torch.cumsum(gone, 0) - gone
        to = torch.where(j < gone[:, None], at[:, None] + j, stack.numel())
        stack = torch.cat((stack, stack[:1])).scatter(0, to.flatten(), seq_pt.flatten())[:-1]
        L, count = torch.where(s["done"] != 0, 0, L), (count + gone.sum()).int()
    have = (L + BK - 1) // BK
    need = (L + n + BK - 1) // BK - have
    off = torch.cumsum(need, 0) - need
    ok = off + need <= count
    cu = torch.cat((torch.zeros_like(n[:1]), torch.cumsum(n, 0))).int()
    i = torch.arange(s["N"], device=L.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=L.numel() - 1)
    live = (i < cu[-1]) & ok[b]
    pos = L[b] + i - cu[b]
    blk = (pos // BK).clamp(max=seq_pt.shape[1] - 1)
    fresh = stack[(count - 1 - (off[b] + blk - have[b])).clamp(min=0, max=stack.numel() - 1)]
    page = torch.where(blk >= have[b], fresh, seq_pt[b, blk]).long()
    given = (j >= have[:, None]) & (j < (have + need)[:, None]) & ok[:, None]
    seq_pt.copy_(torch.where(given, stack[(count - 1 - (off[:, None] + j - have[:, None])).clamp(min=0, max=stack.numel() - 1)], seq_pt))
    return {"seq_len": torch.where(ok, L + n, L).int(), "free_count": (count - (need * ok).sum()).int(), "cu": cu,
            "slot": torch.where(live, page * BK + pos % BK, -1), "pos": torch.where(live, pos, -1).int(),
            "seq": torch.where(live, b, -1).int(), "seq_pt": seq_pt, "free_pages": stack}


def _norm_rotate(x, weight, cos, sin, s):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()
    rot = s["rot"]
    y = x[..., :rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if s["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((u, v), -1).flatten(-2) if s["interleaved"] else torch.cat((u, v), -1)
    return torch.cat((y, x[..., rot:]), -1).bfloat16()


def _plain_rope(s):
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    page, t = s["slots"] // BK, s["slots"] % BK
    s["Q_out"].copy_(_norm_rotate(s["Q"], s["q_weight"], cos, sin, s))
    s["K_pool"][page, :, t] = _norm_rotate(s["K"], s["k_weight"], cos, sin, s)
    if s["V"] is not None:
        s["V_pool"][page, :, t] = s["V"]
    return [s["Q_out"], s["K_pool"], s["V_pool"]]


def _plain_store(s):
    page, t = s["slots"] // BK, s["slots"] % BK
    out = []
    for x, gs in (("K", s["k_scale"]), ("V", s["v_scale"])):
        s[x + "_codes"][page, :, t], s[x + "_scales"][page, :, t] = _quantise(s[x], gs)
        at = s["pages"].long()
        out.append(_values(s[x + "_codes"][at], s[x + "_scales"][at], gs).bfloat16())
    return out


def _plain_sparse(s):
    R, k = s["pt"].shape
    B, Hq, D = s["Q"].shape
    Hkv = R // B
    pages, group = s["pt"].clamp(min=0).long(), (torch.arange(R, device="cuda") % Hkv)[:, None]
    K = _values(s["K_codes"][pages, group], s["K_scales"][pages, group], s["k_scale"]).reshape(R, k * BK, D)
    V = _values(s["V_codes"][pages, group], s["V_scales"][pages, group], s["v_scale"]).reshape(R, k * BK, D)
    z = torch.matmul(s["Q"].float().reshape(R, Hq // Hkv, D), K.transpose(1, 2)) * s["scale"]
    valid = torch.arange(k * BK, device="cuda") < ((s["n"] - 1) * BK + s["last_len"])[:, None]
    z = z.masked_fill(~(valid & (s["n"] > 0)[:, None])[:, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    O = torch.matmul(p, V) / torch.where(l == 0, torch.ones_like(l), l)
    return [O.reshape(B, Hq, D).bfloat16(), (m + torch.log(l)).reshape(B, Hq)]


def _plain_dense(s):
    B, Hq, D = s["Q"].shape
    Hkv = s["K_codes"].shape[1]
    b, j = s["unit_seq"], s["unit_block"]
    pages = s["seq_pt"][b, j].long()
    K = _values(s["K_codes"][pages], s["K_scales"][pages], s["k_scale"])             # [units, Hkv, BK, D]
    q = s["Q"].float().reshape(B, Hkv, Hq // Hkv, D)[b]
    z = torch.matmul(q, K.transpose(2, 3)) * s["scale"]                              # [units, Hkv, G, BK]
    del K
    valid = j[:, None] * BK + torch.arange(BK, device="cuda") < s["seq_len"][b][:, None]
    z = z.masked_fill(~valid[:, None, None], -math.inf)
    shape = (B, Hkv, Hq // Hkv)
    m = torch.full(shape, -math.inf, device="cuda").index_reduce(0, b, z.amax(-1), "amax")
    p = torch.exp(z - m[b][..., None])
    l = torch.zeros(shape, device="cuda").index_add(0, b, p.sum(-1))
    V = _values(s["V_codes"][pages], s["V_scales"][pages], s["v_scale"])
    O = torch.zeros(*shape, D, device="cuda").index_add(0, b, torch.matmul(p, V)) / l[..., None]
    return [O.reshape(B, Hq, D).bfloat16(), (m + torch.log(l)).reshape(B, Hq)]


def run(state):
    s = state
    if own:
        import block_sparse_attention_02_gb300 as msa
        if s["op"] == "tables":
            o, L, count = s["out"], s["seq_len"], s["free_count"]
            if s["any_done"]:
                msa.msa_release_pages(L, s["done"], s["seq_pt"], s["free_pages"], count, o["mid_len"], o["mid_free"],
                                      dev_err=o["err"])
                L, count = o["mid_len"], o["mid_free"]
            msa.msa_plan_step(L, s["new_len"], s["seq_pt"], s["free_pages"], count, o["seq_len"], o["free_count"],
                              o["cu"], o["slot"], o["pos"], o["seq"], num_pages=s["num_pages"], dev_err=o["err"])
            return {"seq_len": o["seq_len"], "free_count": o["free_count"], "cu": o["cu"], "slot": o["slot"],
                    "pos": o["pos"], "seq": o["seq"], "seq_pt": s["seq_pt"], "free_pages": s["free_pages"]}
        if s["op"] == "rope":
            msa.msa_qk_norm_rope(s["Q"], s["K"], s["pos"], s["inv_freq"], s["Q_out"], s["K_pool"], V=s["V"],
                                 V_out=s["V_pool"], slots=s["slots"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                 eps=s["eps"], interleaved=s["interleaved"], dev_err=s["err"])
            return [s["Q_out"], s["K_pool"], s["V_pool"]]
        cache = msa.Q4Cache(s["K_codes"], s["K_scales"], s["V_codes"], s["V_scales"], s["k_scale"], s["v_scale"])
        if s["op"] == "store":
            msa.msa_cache_append_q4(s["K"], s["V"], s["slots"], cache, dev_err=s["err"])
            msa.msa_cache_expand_q4(cache, s["pages"], s["K_out"], s["V_out"], dev_err=s["err"])
            return [s["K_out"], s["V_out"]]
        if s["op"] == "sparse":
            msa.msa_sparse_attn_decode_q4(s["Q"], cache, s["pt"], s["n"], s["last_len"], s["O"], s["LSE"], s["ws"],
                                          dev_err=s["err"], scratch_zeroed=True)
        else:
            msa.msa_dense_attn_decode_q4(s["Q"], cache, s["seq_pt"], s["seq_len"], s["O"], s["LSE"], s["ws"],
                                         dev_err=s["err"], scratch_zeroed=True)
        return [s["O"], s["LSE"]]
    return {"tables": _plain_tables, "rope": _plain_rope, "store": _plain_store, "sparse": _plain_sparse,
            "dense": _plain_dense}[s["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "tables":
        L, n, done = _table_lengths(c)
        pages = sum((a + b + BK - 1) // BK - (a + BK - 1) // BK for a, b in zip(L, n))
        back = sum((a + BK - 1) // BK for a, d in zip(L, done) if d)
        # request lengths in, lengths and offsets out, 16 bytes a token row, a page id moved from the stack or back to it
        return {"bytes": c["B"] * 20 + 16 + 16 * (sum(n) + c["pad"]) + 8 * (pages + back), "flops": 4 * (sum(n) + c["B"])}
    if c["op"] == "rope":
        N, heads = c["N"], c["Hq"] + c["Hkv"]
        moved = heads + (c["Hkv"] if c["values"] else 0)
        return {"bytes": N * moved * c["D"] * 4 + N * 12 + c["D"] * 4 + c["rot"] * 2,
                "flops": N * heads * (4 * c["D"] + 3 * c["rot"])}
    if c["op"] == "store":
        N = c["B"] * c["T"]
        pages = sum(((b * 29 + 1) % BK + c["T"] + BK - 1) // BK for b in range(c["B"]))
        block = c["Hkv"] * BK
        return {"bytes": N * c["Hkv"] * (512 + 144) + N * 8 + pages * block * (144 + 512) + pages * 4,
                "flops": N * c["Hkv"] * 256 * 3 + pages * block * 256}
    if c["op"] == "sparse":
        n, last = _sparse_counts(c)
        tokens = sum((a - 1) * BK + b for a, b in zip(n, last) if a) * c["Hkv"]
        tables = c["B"] * c["Hkv"] * (c["k"] + 2) * 4
    else:
        tokens = sum(_dense_lengths(c)) * c["Hkv"]
        tables = sum((a + BK - 1) // BK for a in _dense_lengths(c)) * 4 + c["B"] * 4
    # a cached token of one KV head: two rows of 64 code bytes and 8 scale bytes
    return {"bytes": tokens * 144 + tables + c["B"] * c["Hq"] * (256 + 256 + 4),
            "flops": tokens * (c["Hq"] // c["Hkv"]) * 4 * 128}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

_E4M3 = [(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127]


def _nearest(grid, x):
    """The value of `grid` (ascending, at places 0, 1, ..) nearest to x >= 0; halfway, the one at the even place."""
    hi = torch.searchsorted(grid, x).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - x, x - grid[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (x >= grid[-1]), grid[hi], grid[lo])


def _exact_round(x, gs):
    f8, f4 = (torch.tensor(v, dtype=torch.float64, device=x.device) for v in (_E4M3, GRID))
    g = x.double().unflatten(-1, (-1, 16))
    step = _nearest(f8, (g.abs().amax(-1, keepdim=True) / 6 / gs).contiguous()) * gs
    v = _nearest(f4, torch.where(step > 0, g.abs() / torch.where(step > 0, step, 1.0), 0.0).contiguous())
    return (torch.sign(g) * v * step).flatten(-2)


def _exact_values(codes, scales, gs):
    low, high = codes.long() & 15, codes.long() >> 4
    f4 = torch.tensor(GRID, dtype=torch.float64, device=codes.device)
    f8 = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device=codes.device)
    c = torch.stack((low, high), -1).flatten(-2)
    v = f4[c & 7] * (1 - 2 * (c >> 3))
    return v * f8[scales.long()].repeat_interleave(16, -1) * gs


def _exact_attend(q, K, V, scale):
    """Output and log-sum-exp of q [G, D] over K, V [T, D]."""
    z = q @ K.T * scale
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[:, None]) @ V, lse


def exact(case, seed):
    if case["op"] == "tables":
        return None                                             # whole numbers: compared as they are
    s = prepare(case, seed)
    if case["op"] == "rope":
        turn = s["pos"].double()[:, None, None] * s["inv_freq"].double()
        out = []
        for x, w in ((s["Q"], s["q_weight"]), (s["K"], s["k_weight"])):
            y = x.double()
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w.double()
            r = y[..., :s["rot"]]
            pair = r.unflatten(-1, (-1, 2)) if s["interleaved"] else r.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.polar(torch.ones_like(turn), turn) * torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous())
            z = torch.view_as_real(z)
            r.copy_((z if s["interleaved"] else z.transpose(-1, -2)).flatten(-2))
            out.append(y)
        pool = torch.zeros(s["K_pool"].shape, dtype=torch.float64, device="cuda")
        flat = pool.transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])
        back = lambda v: flat.index_copy(0, s["slots"], v).unflatten(0, (-1, BK)).transpose(1, 2)  # noqa: E731
        return [out[0], back(out[1]), back(s["V"].double()) if s["V"] is not None else None]
    if case["op"] == "store":
        place = {int(p): i for i, p in enumerate(s["pages"].tolist())}
        at = torch.tensor([place[v // BK] * BK + v % BK for v in s["slots"].tolist()], device="cuda")
        out = []
        for x, gs in (("K", s["k_scale"]), ("V", s["v_scale"])):
            old = _exact_values(s[x + "_codes"], s[x + "_scales"], gs)[s["pages"].long()].transpose(1, 2).flatten(0, 1)
            old = old.index_copy(0, at, _exact_round(s[x], gs))
            out.append(old.unflatten(0, (-1, BK)).transpose(1, 2))
        return out
    B, Hq, D = s["Q"].shape
    Hkv = s["K_codes"].shape[1]
    G = Hq // Hkv
    O = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    LSE = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lengths = s["seq_len"].tolist() if case["op"] == "dense" else None
    counts = list(zip(s["n"].tolist(), s["last_len"].tolist())) if lengths is None else None
    for r in range(B * Hkv):
        b, g = r // Hkv, r % Hkv
        if lengths is not None:
            T = lengths[b]
            pages = s["seq_pt"][b, :(T + BK - 1) // BK].long()
        else:
            n, last = counts[r]
            T = (n - 1) * BK + last
            pages = s["pt"][r, :n].long()
        if pages.numel() == 0:
            continue
        K = _exact_values(s["K_codes"][pages, g], s["K_scales"][pages, g], s["k_scale"]).flatten(0, 1)[:T]
        V = _exact_values(s["V_codes"][pages, g], s["V_scales"][pages, g], s["v_scale"]).flatten(0, 1)[:T]
        h = slice(g * G, (g + 1) * G)
        O[b, h], LSE[b, h] = _exact_attend(s["Q"][b, h].double(), K, V, s["scale"])
    return [O, LSE]
