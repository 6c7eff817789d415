"""Cases of a paged cache held in 8 bits (its store and the decode attention that reads it), of attention through a
sliding window with sinks (prompts, chunks over a paged prefix, single tokens) and of sharing, copying, compacting and
freeing a cache's pages.

Head layout and lengths are those of the framework's workloads (48 query heads over 8 KV heads of 128, 128-token pages,
16 selected pages, 60,001 and 1,048,576 cached tokens, prompts of 131,072 tokens, chunks of 8,192 and of 4 tokens after
60,000 cached ones).  ``own`` chooses between the plain form (elementary torch operations in 32 bits) and the framework's
calls.
"""
import math

import torch

own = False

BK = 128                      # tokens per page
D = 128                       # channels of a head
FIRST, LAST = 87, 167         # scale bytes of the 8-bit cache: 2^(byte - 127), from 2^-40 to 2^40


def listed():
    return [
        # one decoded token for each of 8 sequences into its page, and these pages read back
        dict(name="store8_b8", op="store", B=8, T=1, Hkv=8),
        # a prefill chunk of 8,192 tokens stored, and its pages expanded for the chunk's attention
        dict(name="store8_chunk_t8192", op="store", B=1, T=8192, Hkv=8),
        # decode over the selected pages, 8 sequences
        dict(name="sparse8_b8", op="sparse", B=8, Hq=48, Hkv=8, k=16, short=False),
        # decode over every cached token
        dict(name="dense8_b8_l60001", op="dense", B=8, Hq=48, Hkv=8, lo=60001, hi=60001, window=0, sinks=0, bits=8),
        dict(name="dense8_b1_l1048576", op="dense", B=1, Hq=48, Hkv=8, lo=1048576, hi=1048576, window=0, sinks=0, bits=8),
        # a window layer of a busy server: 64 sequences, most of them longer than the window, one page of sinks
        dict(name="window8_b64", op="dense", B=64, Hq=48, Hkv=8, lo=500, hi=30000, window=4096, sinks=128, bits=8),
        # a window layer's decode over a bf16 cache, a few sinks
        dict(name="window_b8_l60001", op="dense", B=8, Hq=48, Hkv=8, lo=60001, hi=60001, window=2048, sinks=4, bits=16),
        # 4 draft tokens of 8 sequences verified
        dict(name="window_verify_b8_s4", op="window", B=8, S=4, Hq=48, Hkv=8, window=2048, sinks=4, paged=True, lo=60000,
             hi=60000),
        # a prefill chunk after a cached prefix
        dict(name="window_chunk_s8192", op="window", B=1, S=8192, Hq=48, Hkv=8, window=4096, sinks=4, paged=True, lo=60000,
             hi=60000),
        # a window layer over a whole prompt
        dict(name="window_s131072", op="window", B=1, S=131072, Hq=48, Hkv=8, window=2048, sinks=128, paged=False, lo=0,
             hi=0),
        # parallel sampling: of 64 running samples 24 end, and 8 of the others are continued in these rows three times each
        dict(name="fork_b64", op="fork", B=64, done=24, shared=30, forks=24, pad=8, lo=2000, hi=20000, Hkv=8),
        # a pool of 2,048 pages, half of them in use, gathered at its front
        dict(name="compact_p2048", op="compact", B=24, lo=500, hi=20000, shared=20, pool=2048, Hkv=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["store", "store", "sparse", "dense", "dense", "dense", "window", "window", "window", "fork", "compact"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op == "store":
        T = _log(rng, 1, 8192)
        return dict(op=op, B=_log(rng, 1, max(1, min(128, 8192 // T))), T=T, Hkv=Hkv)
    if op == "sparse":
        return dict(op=op, B=_log(rng, 1, 128), Hq=Hq, Hkv=Hkv, k=rng.choice([1, 4, 8, 16, 16, 24, 32]), short=rng.random() < 0.5)
    if op == "dense":
        bits = rng.choice([8, 8, 16])
        windowed = bits == 16 or rng.random() < 0.4
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 1000000 // B))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, lo=_log(rng, 1, hi), hi=hi, window=_log(rng, 1, 8192) if windowed else 0,
                    sinks=rng.choice([0, 1, 4, 64, 128, 300]) if windowed else 0, bits=bits)
    if op == "window":
        paged = rng.random() < 0.6
        window = _log(rng, 1, 8192)
        B = _log(rng, 1, 16)
        S = _log(rng, 1, max(1, min(65536, 100000000 // window) // B))
        hi = _log(rng, 1, 65536) if paged else 0
        return dict(op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, window=window, sinks=rng.choice([0, 1, 4, 64, 128, 300]), paged=paged,
                    lo=_log(rng, 1, hi) if paged else 0, hi=hi)
    B = _log(rng, 2, 512)
    hi = _log(rng, 1, max(1, 200000 // B))
    lo = _log(rng, 1, hi)
    shared = rng.randint(0, 60)
    if op == "fork":
        done = rng.randint(1, max(1, B // 2))
        return dict(op=op, B=B, done=done, shared=shared, forks=rng.randint(1, done), pad=rng.choice([0, 1, 9]), lo=lo, hi=hi, Hkv=Hkv)
    return dict(op=op, B=B, lo=lo, hi=hi, shared=shared, pool=_log(rng, 64, 2048) + B * (hi // BK + 1), Hkv=Hkv)


# ---------------------------------------------------------------------------
# sizes that follow from a case alone
# ---------------------------------------------------------------------------

def _spread(n, lo, hi, turn):
    """n lengths over [lo, hi], evenly on a logarithmic scale, in an order of their own."""
    if lo >= hi:
        return [lo] * n
    return [max(lo, min(hi, int(lo * (hi / lo) ** ((((i * 37 + turn) % n) + 0.5) / n)))) for i in range(n)]


def _pages(tokens):
    return (tokens + BK - 1) // BK


def _store_starts(c):
    """Tokens that each sequence's first page holds already."""
    return [(b * 29 + 1) % BK for b in range(c["B"])]


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


def _seen(L, window, sinks):
    """Of a query at the end of L tokens: the first token of its window (0: everything), and the sinks before it."""
    first = max(0, L - window) if window else 0
    return first, min(sinks, first)


def _dense_lengths(c):
    return _spread(c["B"], c["lo"], c["hi"], 1)


def _seen_pages(L, c):
    """The pages of a sequence that hold a token its query sees."""
    first, sinks = _seen(L, c["window"], c["sinks"])
    return sorted(set(range(_pages(sinks))) | set(range(first // BK, _pages(L))))


def _prefixes(c):
    return _spread(c["B"], c["lo"], c["hi"], 2) if c["paged"] else [0] * c["B"]


def _window_keys(c):
    """Keys seen, summed over the queries of all sequences."""
    W, n = c["window"], 0
    for p in _prefixes(c):
        # query i (from p on) sees min(i + 1, W) tokens of its window and min(sinks, i + 1 - W) before it
        def upto(m, top):                                        # sum over i < m of min(i + 1, top)
            return m * (m + 1) // 2 if m <= top else top * (top + 1) // 2 + (m - top) * top
        n += upto(p + c["S"], W) - upto(p, W)
        if c["sinks"]:
            n += upto(max(0, p + c["S"] - W), c["sinks"]) - upto(max(0, p - W), c["sinks"])
    return n


def _requests(c):
    """(lengths, page tables as lists of pool pages, pages in use) of B requests, some of which share their first pages."""
    L = _spread(c["B"], c["lo"], c["hi"], 5)
    tables, nxt = [], 0
    for b, x in enumerate(L):
        n = _pages(x)
        common = 0
        if b > 0 and (b * 61) % 100 < c["shared"]:               # a fork of the request before: its full pages, as far as both have them
            common = min(x, L[b - 1]) // BK
        tables.append(tables[-1][:common] + list(range(nxt, nxt + n - common)) if b else list(range(n)))
        nxt += n - common
    return L, tables, nxt


def _turnover(c):
    """(requests that end, requests that are continued in the first of their rows, three times each)."""
    gone = [b for b in range(c["B"]) if b * c["done"] // c["B"] != (b + 1) * c["done"] // c["B"]]
    kept = [b for b in range(c["B"]) if b not in gone]
    return gone, [kept[i // 3 % len(kept)] for i in range(c["forks"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _bf16(g, *shape, scale=1.0):
    """Normal values, drawn in parts so that no large tensor of 32 bits stands beside them."""
    x = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    for part in x.view(-1).split(1 << 28):
        part.copy_(_normal(g, part.numel()) * scale)
    return x


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _fill_cache(g, pages, Hkv):
    """An 8-bit cache of normal keys (some channels larger, as trained keys have) and values, blocks of differing size."""
    chan = torch.exp(0.4 * _normal(g, Hkv, 1, D))
    c = {}
    for side in ("K", "V"):
        codes = torch.empty(pages, Hkv, BK, D, dtype=torch.uint8, device="cuda")
        scales = torch.empty(pages, Hkv, dtype=torch.uint8, device="cuda")
        for p in range(0, pages, 1024):
            n = min(1024, pages - p)
            x = _normal(g, n, Hkv, BK, D) * torch.exp(0.5 * _normal(g, n, Hkv, 1, 1))
            x = (x * chan if side == "K" else x).bfloat16().float()
            scales[p:p + n] = _scale_byte(x.abs().amax((-1, -2)))
            codes[p:p + n] = _encode(x, scales[p:p + n, :, None, None])
        c[side + "_codes"], c[side + "_scales"] = codes, scales
    return c


def _tables(tables, width, ids):
    """Page tables as a tensor, -1 past each request's pages, page i of the lists being ids[i]."""
    t = torch.full((len(tables), width), -1, dtype=torch.int32)
    ids = ids.cpu()
    for b, row in enumerate(tables):
        t[b, :len(row)] = ids[torch.tensor(row, dtype=torch.long)]
    return t.cuda()


def prepare(case, seed):
    g = _gen(seed)
    op, Hkv = case["op"], case["Hkv"]
    s = {"err": _ints([0])}
    if op == "store":
        B, T = case["B"], case["T"]
        start = _store_starts(case)
        per = [_pages(a + T) for a in start]
        pages = torch.randperm(sum(per), generator=g, device="cuda").int()
        first = [sum(per[:b]) for b in range(B)]
        at = torch.cat([torch.arange(a, a + T) + f * BK for a, f in zip(start, first)]).cuda()
        chan = torch.exp(0.4 * _normal(g, Hkv, D))
        size = torch.exp(0.5 * _normal(g, B * T, 1, 1))          # tokens of differing size: some make their block's scale grow
        s |= _fill_cache(g, sum(per), Hkv)
        s |= {"K": (_normal(g, B * T, Hkv, D) * chan * size).bfloat16(), "V": (_normal(g, B * T, Hkv, D) * size).bfloat16(),
              "slots": pages[at // BK].long() * BK + at % BK, "pages": pages}
        for x in ("K", "V"):
            s[x + "_out"] = torch.empty(sum(per), Hkv, BK, D, dtype=torch.bfloat16, device="cuda")
    elif op in ("sparse", "dense"):
        B, Hq = case["B"], case["Hq"]
        s |= {"Q": (1.5 * _normal(g, B, Hq, D)).bfloat16(), "scale": 1 / math.sqrt(D)}
        if op == "sparse":
            k = case["k"]
            n, last = _sparse_counts(case)
            pool = max(B * k * 2, 64)                            # a cache that holds more than the selected pages
            pick = torch.rand(B * Hkv, pool // B, generator=g, device="cuda").argsort(1)[:, :k] \
                + (torch.arange(B * Hkv, device="cuda") // Hkv * (pool // B))[:, None]
            live = torch.arange(k, device="cuda") < _ints(n).repeat_interleave(Hkv)[:, None]
            s |= {"pt": torch.where(live, pick, torch.full_like(pick, -1)).int(), "n": _ints(n).repeat_interleave(Hkv),
                  "last_len": _ints(last).repeat_interleave(Hkv), "k": k}
        else:
            L = _dense_lengths(case)
            per = [_pages(a) for a in L]
            pool = sum(per)
            ids = torch.randperm(pool, generator=g, device="cuda")
            firsts = [sum(per[:b]) for b in range(B)]
            seen = [_seen_pages(x, case) for x in L]
            s |= {"seq_pt": _tables([list(range(f, f + n)) for f, n in zip(firsts, per)], max(per), ids), "seq_len": _ints(L),
                  "window": case["window"], "sinks": case["sinks"],
                  # which (sequence, block) each page that is seen is, as the program's scheduler knows it
                  "unit_seq": torch.repeat_interleave(torch.arange(B), torch.tensor([len(x) for x in seen])).cuda(),
                  "unit_block": torch.tensor([j for x in seen for j in x]).cuda()}
        if op == "dense" and case["bits"] == 16:
            s |= {"K_pool": _bf16(g, pool, Hkv, BK, D), "V_pool": _bf16(g, pool, Hkv, BK, D)}
        else:
            s |= _fill_cache(g, pool, Hkv)
        s["O"] = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["LSE"] = torch.empty(B, Hq, dtype=torch.float32, device="cuda")
        # scratch, as a program keeps it: zero-filled, and large enough for any split of the work
        s["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    elif op == "window":
        B, S, Hq = case["B"], case["S"], case["Hq"]
        s |= {"Q": _bf16(g, B, S, Hq, D, scale=1.5), "scale": 1 / math.sqrt(D), "window": case["window"], "sinks": case["sinks"]}
        if case["paged"]:
            pos = _prefixes(case)
            per = [_pages(p + S) for p in pos]
            ids = torch.randperm(sum(per), generator=g, device="cuda")
            firsts = [sum(per[:b]) for b in range(B)]
            s |= {"K": _bf16(g, sum(per), Hkv, BK, D), "V": _bf16(g, sum(per), Hkv, BK, D), "q_pos": _ints(pos),
                  "seq_pt": _tables([list(range(f, f + n)) for f, n in zip(firsts, per)], max(per), ids), "first": min(pos)}
        else:
            s |= {"K": _bf16(g, B, S, Hkv, D), "V": _bf16(g, B, S, Hkv, D), "q_pos": None, "seq_pt": None, "first": 0}
        s["O"] = torch.empty(B, S, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["LSE"] = torch.empty(B, S, Hq, dtype=torch.float32, device="cuda")
    else:
        L, tables, used = _requests(case)
        B = len(L)
        pool = used + B + 16 if op == "fork" else max(case["pool"], used)
        ids = torch.randperm(pool, generator=g, device="cuda").int()
        width = max(_pages(max(L)) + 1, 4)
        times = torch.zeros(pool, dtype=torch.int32)
        for row in tables:
            times[torch.tensor(row, dtype=torch.long)] += 1
        shares = torch.zeros(pool, dtype=torch.int32, device="cuda")
        shares[ids.long()] = (times - 1).clamp(min=0).cuda()      # requests that hold a page besides its first one
        free = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        free[:pool - used] = ids[used:]
        s |= {"seq_len": _ints(L), "seq_pt": _tables(tables, width, ids), "shares": shares, "free": free,
              "free_count": _ints([pool - used]), "shares_out": torch.empty_like(shares), "count_out": _ints([0]),
              # the cache of one layer: keys, values, index keys
              "pools": [_bf16(g, pool, Hkv, BK, D), _bf16(g, pool, Hkv, BK, D), _bf16(g, pool, Hkv, BK, D // 2)]}
        if op == "fork":
            gone, src = _turnover(case)
            dst, pad = gone[:len(src)], case["pad"]              # padded to the rows of a captured graph
            F = len(src) + pad
            s |= {"done": _ints([int(b in gone) for b in range(B)]), "src": _ints(src + [-1] * pad), "dst": _ints(dst + [-1] * pad),
                  "mid_len": torch.empty(B, dtype=torch.int32, device="cuda"), "mid_count": _ints([0]),
                  "mid_shares": torch.empty_like(shares), "len_out": torch.empty(B, dtype=torch.int32, device="cuda"),
                  "copy_src": torch.empty(F, dtype=torch.int32, device="cuda"),
                      "copy_dst": torch.empty(F, dtype=torch.int32, device="cuda"), "pt_out": s["seq_pt"].clone()}
        else:
            s |= {"pt_out": torch.full_like(s["seq_pt"], -1), "free_out": torch.empty_like(free),
                  "move_src": torch.empty(pool, dtype=torch.int32, device="cuda"),
                  "move_dst": torch.empty(pool, dtype=torch.int32, device="cuda")}
    s["op"] = op
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _scale_byte(amax):
    """The byte of the smallest power of two, from 2^-40 to 2^40, that amax is at most 448 times of."""
    fraction, exponent = torch.frexp(amax)                       # amax = fraction * 2^exponent, 448 = 0.875 * 2^9
    e = exponent - 9 + (fraction > 0.875).int()
    return torch.where(amax > 0, e + 127, torch.full_like(e, FIRST)).clamp(FIRST, LAST).to(torch.uint8)


def _power(byte):
    return (byte.int().clamp(FIRST, LAST) << 23).view(torch.float32)          # the byte is a float's exponent: no power function's rounding


def _encode(x, byte):
    return (x / _power(byte)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, byte):
    """What blocks [.., BK, D] of codes stand for, in 32 bits; byte [..]."""
    return codes.view(torch.float8_e4m3fn).float() * _power(byte)[..., None, None]


def _plain_store(s):
    page, t, at = s["slots"] // BK, s["slots"] % BK, s["pages"].long()
    place = torch.empty_like(at).scatter_(0, at, torch.arange(at.numel(), device=at.device))[page]
    # rows before it stay, with their block's scale; what lies behind the last new one is of no sequence and keeps its codes
    r0 = torch.full_like(at, BK).scatter_reduce(0, place, t, "amin")
    out = []
    for x in ("K", "V"):
        new = s[x].float()
        amax = torch.zeros(at.numel(), new.shape[1], device=at.device)
        amax = amax.scatter_reduce(0, place[:, None].expand(-1, new.shape[1]), new.abs().amax(-1), "amax")
        codes, old = s[x + "_codes"][at], s[x + "_scales"][at]
        byte = torch.where((r0 > 0)[:, None], torch.maximum(old, _scale_byte(amax)), _scale_byte(amax))
        byte = torch.where((r0 < BK)[:, None], byte, old)
        stays = ((torch.arange(BK, device=at.device) < r0[:, None])[:, None] & (byte != old)[..., None])[..., None]
        codes = torch.where(stays, _encode(_values(codes, old), byte[..., None, None]), codes)
        codes[place, :, t] = _encode(new, byte[place][..., None])
        s[x + "_codes"][at], s[x + "_scales"][at] = codes, byte
        out.append(_values(codes, byte).bfloat16())
    return out


def _softmax_parts(z):
    m = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    return m, p, p.sum(-1, keepdim=True)


def _plain_sparse(s):
    R, k = s["pt"].shape
    B, Hq, _ = s["Q"].shape
    Hkv = R // B
    pages, group = s["pt"].clamp(min=0).long(), (torch.arange(R, device="cuda") % Hkv)[:, None]
    K = _values(s["K_codes"][pages, group], s["K_scales"][pages, group]).reshape(R, k * BK, D)
    V = _values(s["V_codes"][pages, group], s["V_scales"][pages, group]).reshape(R, k * BK, D)
    z = torch.matmul(s["Q"].float().reshape(R, Hq // Hkv, D), K.transpose(1, 2)) * s["scale"]
    valid = torch.arange(k * BK, device="cuda") < ((s["n"] - 1) * BK + s["last_len"])[:, None]
    m, p, l = _softmax_parts(z.masked_fill(~(valid & (s["n"] > 0)[:, None])[:, None], -math.inf))
    O = torch.matmul(p, V) / torch.where(l == 0, torch.ones_like(l), l)
    return [O.reshape(B, Hq, D).bfloat16(), (m + torch.log(l)).reshape(B, Hq)]


def _plain_dense(s):
    B, Hq, _ = s["Q"].shape
    b, j = s["unit_seq"], s["unit_block"]
    pages = s["seq_pt"][b, j].long()
    if "K_pool" in s:
        K, V = s["K_pool"][pages].float(), s["V_pool"][pages].float()
    else:
        K, V = (_values(s[x + "_codes"][pages], s[x + "_scales"][pages]) for x in ("K", "V"))
    Hkv = K.shape[1]
    q = s["Q"].float().reshape(B, Hkv, Hq // Hkv, D)[b]
    z = torch.matmul(q, K.transpose(2, 3)) * s["scale"]                       # [units, Hkv, G, BK]
    L = s["seq_len"][b][:, None]
    t = j[:, None] * BK + torch.arange(BK, device="cuda")
    valid = t < L
    if s["window"]:
        valid &= (t >= L - s["window"]) | (t < s["sinks"])
    z = z.masked_fill(~valid[:, None, None], -math.inf)
    shape = (B, Hkv, Hq // Hkv)
    m = torch.full(shape, -math.inf, device="cuda").index_reduce(0, b, z.amax(-1), "amax")
    p = torch.exp(z - m[b][..., None])
    l = torch.zeros(shape, device="cuda").index_add(0, b, p.sum(-1))
    O = torch.zeros(*shape, D, device="cuda").index_add(0, b, torch.matmul(p, V)) / l[..., None]
    return [O.reshape(B, Hq, D).bfloat16(), (m + torch.log(l)).reshape(B, Hq)]


def _plain_window(s):
    """Blocks of queries, each against its window's tokens and the sinks before them, side by side."""
    B, S, Hq, _ = s["Q"].shape
    W, sinks, first = s["window"], s["sinks"], s["first"]
    Hkv = s["K"].shape[1] if s["q_pos"] is not None else s["K"].shape[2]
    blk = min(BK, S)
    n = (S + blk - 1) // blk
    start = (s["q_pos"].long()[:, None] if s["q_pos"] is not None else torch.zeros(B, 1, dtype=torch.long, device="cuda")) \
        + torch.arange(n, device="cuda") * blk                                # position of each block's first query
    i = start[..., None] + torch.arange(blk, device="cuda")                   # [B, n, blk]
    width = blk + W - 1
    t = start[..., None] - (W - 1) + torch.arange(width, device="cuda")       # [B, n, width]
    t = torch.cat((torch.arange(sinks, device="cuda").expand(B, n, sinks), t), -1)
    last = start[:, :1] + (S - 1)
    seen = (t[:, :, None] <= i[..., None]) & (t[:, :, None] >= 0)
    seen &= torch.where(torch.arange(sinks + width, device="cuda") < sinks, t[:, :, None] <= i[..., None] - W, t[:, :, None] > i[..., None] - W)
    t = torch.minimum(t.clamp(min=0), last[..., None])
    row = torch.arange(B, device="cuda")[:, None, None]

    def take(x):                                                              # [B, n, Hkv, keys, D]
        if s["q_pos"] is None:
            y = x[row, t]
        else:
            y = x[s["seq_pt"][row, t // BK].long(), :, t % BK]
        return y.float().transpose(2, 3)

    q = torch.nn.functional.pad(s["Q"].float(), (0, 0, 0, 0, 0, n * blk - S)).reshape(B, n, blk, Hkv, Hq // Hkv, D)
    q = q.permute(0, 1, 3, 4, 2, 5).reshape(B, n, Hkv, Hq // Hkv * blk, D)
    z = torch.matmul(q, take(s["K"]).transpose(3, 4)).mul_(s["scale"])
    z = z.unflatten(3, (Hq // Hkv, blk)).masked_fill_(~seen[:, :, None, None], -math.inf).flatten(3, 4)
    m, p, l = _softmax_parts(z)
    O = torch.matmul(p, take(s["V"])).div_(l)
    back = lambda x: x.unflatten(3, (Hq // Hkv, blk)).permute(0, 1, 4, 2, 3, 5).reshape(B, n * blk, Hq, -1)[:, :S]  # noqa: E731
    return [back(O).bfloat16(), back(m + torch.log(l))[..., 0].contiguous()]


def _plain_release(s):
    """Ended requests give up their pages; those that none holds any more go back on the stack, by their number."""
    L, pt = s["seq_len"], s["seq_pt"]
    j = torch.arange(pt.shape[1], device=L.device)
    held = (j < ((L + BK - 1) // BK)[:, None]) & (s["done"] != 0)[:, None]
    pool = s["shares"].numel()
    times = torch.zeros(pool + 1, dtype=torch.int32, device=L.device)
    times = times.index_add(0, torch.where(held, pt, pool).flatten().long(), torch.ones_like(pt).flatten())[:pool]
    left = s["shares"] - times
    back = left < 0
    at = torch.where(back, s["free_count"] + torch.cumsum(back, 0) - 1, pool)
    free = torch.cat((s["free"], s["free"][:1])).scatter(0, at, torch.arange(pool, dtype=torch.int32, device=L.device))[:-1]
    return torch.where(s["done"] != 0, 0, L), free, (s["free_count"] + back.sum()).int(), left.clamp(min=0)


def _plain_fork(s):
    L, free, count, shares = _plain_release(s)
    live = s["src"] >= 0
    src, dst = s["src"].clamp(min=0).long(), s["dst"].long()
    n = torch.where(live, L[src], 0)
    full, tail = n // BK, (n % BK > 0)
    order = torch.cumsum(tail, 0) - tail.int()
    page = free[(count - 1 - order).clamp(min=0)]
    pt = torch.cat((s["seq_pt"], s["seq_pt"][:1]))                             # the row after the last takes what is left out
    j = torch.arange(pt.shape[1], device=L.device)
    common = j < full[:, None]
    rows = torch.where(common, pt[src], pt[dst])
    rows = torch.where((j == full[:, None]) & tail[:, None], page[:, None], rows)
    to = torch.where(live, dst, L.numel())
    copy_src, copy_dst = torch.where(tail, pt[src, full.long()], -1).int(), torch.where(tail, page, -1).int()
    s["pt_out"].copy_(pt.index_copy(0, to, rows)[:-1])
    pool = shares.numel()
    shares = torch.cat((shares, shares[:1])).index_add(0, torch.where(common & live[:, None], pt[src], pool).flatten().long(),
                                                       torch.ones_like(rows).flatten())[:pool]
    L = torch.cat((L, L[:1])).index_copy(0, to, n)[:-1]
    _plain_copy(s, copy_src, copy_dst)
    return {"seq_len": L, "seq_pt": s["pt_out"], "free": free, "free_count": (count - tail.sum()).int(), "shares": shares,
            "copy_src": copy_src, "copy_dst": copy_dst, "pools": s["pools"]}


def _plain_copy(s, src, dst):
    keep = src >= 0
    for x in s["pools"]:
        x[dst[keep].long()] = x[src[keep].long()]


def _plain_compact(s):
    L, pt, pool = s["seq_len"], s["seq_pt"], s["shares"].numel()
    j = torch.arange(pt.shape[1], device=L.device)
    held = j < ((L + BK - 1) // BK)[:, None]
    live = torch.zeros(pool + 1, dtype=torch.bool, device=L.device).index_fill(0, torch.where(held, pt, pool).flatten().long(), True)[:pool]
    n = live.sum()
    at = torch.arange(pool, device=L.device)
    goes, hole = live & (at >= n), ~live & (at < n)
    rank = torch.where(goes, torch.cumsum(goes, 0) - 1, torch.where(hole, torch.cumsum(hole, 0) - 1, pool))
    src = torch.full((pool + 1,), -1, dtype=torch.int32, device=L.device).scatter(0, torch.where(goes, rank, pool), at.int())
    dst = torch.full((pool + 1,), -1, dtype=torch.int32, device=L.device).scatter(0, torch.where(hole, rank, pool), at.int())
    src[pool], dst[pool] = -1, -1
    moved = torch.where(goes, dst[rank], at.int())
    s["pt_out"].copy_(torch.where(held, moved[pt.clamp(min=0).long()], s["pt_out"]))
    shares = torch.zeros_like(s["shares"]).scatter_add(0, torch.where(live, moved, pool - 1).long(), torch.where(live, s["shares"], 0))
    free = torch.where(at < pool - n, pool - 1 - at, -1).int()
    _plain_copy(s, src[:pool], dst[:pool])
    return {"seq_pt": s["pt_out"], "shares": shares, "free": free, "free_count": (pool - n).reshape(1).int(), "move_src": src[:pool],
            "move_dst": dst[:pool], "pools": s["pools"]}


def run(state):
    s = state
    if own:
        import block_sparse_attention_02_gb300 as msa
        e = s["err"]
        if s["op"] == "window":
            msa.msa_window_attn_prefill(s["Q"], s["K"], s["V"], s["O"], s["LSE"], window=s["window"], sinks=s["sinks"],
                                        seq_pt=s["seq_pt"], q_pos=s["q_pos"], dev_err=e)
            return [s["O"], s["LSE"]]
        if s["op"] == "fork":
            msa.msa_release_shared_pages(s["seq_len"], s["done"], s["seq_pt"], s["free"], s["free_count"], s["shares"],
                                         s["mid_len"], s["mid_count"], s["mid_shares"], dev_err=e)
            msa.msa_fork_requests(s["src"], s["dst"], s["mid_len"], s["seq_pt"], s["free"], s["mid_count"], s["mid_shares"],
                                  s["len_out"], s["pt_out"], s["count_out"], s["shares_out"], s["copy_src"], s["copy_dst"],
                                  dev_err=e)
            msa.msa_copy_pages(s["pools"], s["copy_src"], s["copy_dst"], dev_err=e)
            return {"seq_len": s["len_out"], "seq_pt": s["pt_out"], "free": s["free"], "free_count": s["count_out"],
                    "shares": s["shares_out"], "copy_src": s["copy_src"], "copy_dst": s["copy_dst"], "pools": s["pools"]}
        if s["op"] == "compact":
            msa.msa_compact_pages(s["seq_len"], s["seq_pt"], s["shares"], s["pt_out"], s["shares_out"], s["free_out"],
                                  s["count_out"], s["move_src"], s["move_dst"], dev_err=e)
            msa.msa_copy_pages(s["pools"], s["move_src"], s["move_dst"], dev_err=e)
            return {"seq_pt": s["pt_out"], "shares": s["shares_out"], "free": s["free_out"], "free_count": s["count_out"],
                    "move_src": s["move_src"], "move_dst": s["move_dst"], "pools": s["pools"]}
        if "K_pool" in s:
            msa.msa_window_attn_decode(s["Q"], s["K_pool"], s["V_pool"], s["seq_pt"], s["seq_len"], s["O"], s["LSE"], s["ws"],
                                       window=s["window"], sinks=s["sinks"], dev_err=e, scratch_zeroed=True)
            return [s["O"], s["LSE"]]
        cache = msa.Q8Cache(s["K_codes"], s["K_scales"], s["V_codes"], s["V_scales"])
        if s["op"] == "store":
            msa.msa_cache_append_q8(s["K"], s["V"], s["slots"], cache, dev_err=e)
            msa.msa_cache_expand_q8(cache, s["pages"], s["K_out"], s["V_out"], dev_err=e)
            return [s["K_out"], s["V_out"]]
        if s["op"] == "sparse":
            msa.msa_sparse_attn_decode_q8(s["Q"], cache, s["pt"], s["n"], s["last_len"], s["O"], s["LSE"], s["ws"], dev_err=e,
                                          scratch_zeroed=True)
        else:
            msa.msa_dense_attn_decode_q8(s["Q"], cache, s["seq_pt"], s["seq_len"], s["O"], s["LSE"], s["ws"],
                                         window=s["window"], sinks=s["sinks"], dev_err=e, scratch_zeroed=True)
        return [s["O"], s["LSE"]]
    return {"store": _plain_store, "sparse": _plain_sparse, "dense": _plain_dense, "window": _plain_window, "fork": _plain_fork,
            "compact": _plain_compact}[s["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c, Hkv = case, case["Hkv"]
    if c["op"] == "store":
        N = c["B"] * c["T"]
        pages = sum(_pages(a + c["T"]) for a in _store_starts(c))
        # tokens in, their codes out; then every page's codes in and its values out
        return {"bytes": N * Hkv * (512 + 256) + N * 8 + pages * (Hkv * (BK * (256 + 512) + 2) + 4), "flops": N * Hkv * 256 * 3 + pages * Hkv * BK * 256}
    if c["op"] in ("sparse", "dense"):
        if c["op"] == "sparse":
            n, last = _sparse_counts(c)
            tokens, pages = sum((a - 1) * BK + b for a, b in zip(n, last) if a), sum(n)
            tables, bits = c["B"] * Hkv * (c["k"] + 2) * 4, 8
        else:
            L = _dense_lengths(c)
            seen = [_seen(x, c["window"], c["sinks"]) for x in L]
            tokens, pages = sum(x - a + b for x, (a, b) in zip(L, seen)), sum(len(_seen_pages(x, c)) for x in L)
            tables, bits = pages * 4 + c["B"] * 4, c["bits"]
        # a cached token of one KV head: two rows of 128 values
        return {"bytes": tokens * Hkv * D * bits // 4 + pages * Hkv * (2 if bits == 8 else 0) + tables + c["B"] * c["Hq"] * (256 + 256 + 4),
                "flops": tokens * c["Hq"] * 4 * D}
    if c["op"] == "window":
        reach = 0                                                             # cached tokens that some query sees
        for p in _prefixes(c):
            first, sinks = _seen(p + 1, c["window"], c["sinks"])
            end = p + c["S"]
            reach += end - first + min(c["sinks"], first)
        return {"bytes": c["B"] * c["S"] * c["Hq"] * (256 + 256 + 4) + reach * Hkv * 512, "flops": _window_keys(c) * c["Hq"] * 4 * D}
    L, tables, used = _requests(c)
    page = Hkv * BK * (D + D + D // 2) * 2
    if c["op"] == "fork":
        B, pool = len(L), used + len(L) + 16
        gone, src = _turnover(c)
        tails = sum(L[b] % BK > 0 for b in src)
        entries = sum(_pages(L[b]) for b in gone) + 2 * sum(L[b] // BK for b in src)
        return {"bytes": 2 * tails * page + 4 * (entries + 2 * pool + 5 * B + 4 * len(src)), "flops": entries}
    pool = max(c["pool"], used)
    moves = used * (pool - used) // pool                                       # of pages anywhere in the pool, this share lies behind the first `used`
    return {"bytes": 2 * moves * page + 4 * (2 * sum(_pages(x) for x in L) + 5 * pool), "flops": pool}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

_E4M3 = [(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127]


def _exact_power(byte):
    return torch.tensor([2.0 ** (e - 127) for e in range(FIRST, LAST + 1)], dtype=torch.float64, device=byte.device)[byte.long().clamp(FIRST, LAST) - FIRST]


def _exact_values(codes, byte):
    f8 = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device=codes.device)
    v = f8[(codes & 127).long()] * (1 - 2 * (codes >> 7).double())
    return v * _exact_power(byte)


def _exact_round(x, step):
    """x (64 bits) to the nearest of step * the 8-bit float's values; halfway, the one with the even code."""
    grid = torch.tensor(_E4M3, dtype=torch.float64, device=x.device)
    a = (x.abs() / step).contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    return torch.sign(x) * torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (a >= grid[-1]), grid[hi], grid[lo]) * step


def _exact_store(s):
    pages, slots = s["pages"].tolist(), s["slots"]
    page_of = (slots // BK).tolist()
    rows = {}
    for r, p in enumerate(page_of):
        rows.setdefault(p, []).append(r)
    out = []
    for x in ("K", "V"):
        blocks = []
        for p in pages:
            v = _exact_values(s[x + "_codes"][p], s[x + "_scales"][p][:, None, None])               # [Hkv, BK, D]
            if p in rows:
                at = torch.tensor(rows[p], device="cuda")
                t, new = slots[at] % BK, s[x][at].double().transpose(0, 1)                             # [Hkv, rows, D]
                powers = _exact_power(torch.arange(FIRST, LAST + 1, device="cuda"))
                step = powers[torch.searchsorted(powers, new.abs().amax((1, 2)) / 448).clamp(max=LAST - FIRST)]
                old, n = _exact_power(s[x + "_scales"][p]), int(t.min())
                if n > 0:
                    step = torch.where(step > old, step, old)
                    v[:, :n] = torch.where((step > old)[:, None, None], _exact_round(v[:, :n], step[:, None, None]), v[:, :n])
                v[:, n:] *= (step / old)[:, None, None]          # codes as they are, of another scale
                v[:, t] = _exact_round(new, step[:, None, None])
            blocks.append(v)
        out.append(torch.stack(blocks))
    return out


def _exact_attend(q, K, V, scale, seen=None):
    """Output and log-sum-exp of q [.., D] over K, V [T, D]."""
    z = q @ K.T * scale
    if seen is not None:
        z = z.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[..., None]) @ V, lse


def _exact_decode(case, s):
    B, Hq, _ = s["Q"].shape
    Hkv = case["Hkv"]
    G = Hq // Hkv
    O = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    LSE = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lengths = s["seq_len"].tolist() if case["op"] == "dense" else None
    counts = list(zip(s["n"].tolist(), s["last_len"].tolist())) if lengths is None else None
    for r in range(B * Hkv):
        b, g = r // Hkv, r % Hkv
        if lengths is not None:
            T = lengths[b]
            first, sinks = _seen(T, case["window"], case["sinks"])
            tokens = torch.cat((torch.arange(sinks, device="cuda"), torch.arange(first, T, device="cuda")))
            pages = s["seq_pt"][b, tokens // BK].long()
        else:
            n, last = counts[r]
            tokens = torch.arange((n - 1) * BK + last if n else 0, device="cuda")
            pages = s["pt"][r, tokens // BK].long()
        if tokens.numel() == 0:
            continue
        at = tokens % BK
        if "K_pool" in s:
            K, V = s["K_pool"][pages, g, at].double(), s["V_pool"][pages, g, at].double()
        else:
            K, V = (_exact_values(s[x + "_codes"][pages, g, at], s[x + "_scales"][pages, g][:, None]) for x in ("K", "V"))
        h = slice(g * G, (g + 1) * G)
        O[b, h], LSE[b, h] = _exact_attend(s["Q"][b, h].double(), K, V, s["scale"])
    return [O, LSE]


def _exact_window(case, s):
    B, S, Hq, _ = s["Q"].shape
    Hkv, W, sinks = case["Hkv"], case["window"], case["sinks"]
    G, step = Hq // Hkv, 512
    O = torch.empty(B, S, Hq, D, dtype=torch.float64, device="cuda")
    LSE = torch.empty(B, S, Hq, dtype=torch.float64, device="cuda")
    for b, p in enumerate(_prefixes(case)):
        for g in range(Hkv):
            if case["paged"]:
                pages = s["seq_pt"][b, :_pages(p + S)].long()
                K, V = s["K"][pages, g].flatten(0, 1), s["V"][pages, g].flatten(0, 1)
            else:
                K, V = s["K"][b, :, g], s["V"][b, :, g]
            for lo in range(0, S, step):
                i = p + torch.arange(lo, min(lo + step, S), device="cuda")
                first = max(0, p + lo - W + 1)
                t = torch.cat((torch.arange(min(sinks, first), device="cuda"), torch.arange(first, int(i[-1]) + 1, device="cuda")))
                seen = (t <= i[:, None]) & ((t > i[:, None] - W) | (t < sinks))
                q = s["Q"][b, lo:lo + step, g * G:(g + 1) * G].double().transpose(0, 1)
                o, l = _exact_attend(q, K[t].double(), V[t].double(), s["scale"], seen)
                O[b, lo:lo + step, g * G:(g + 1) * G], LSE[b, lo:lo + step, g * G:(g + 1) * G] = o.transpose(0, 1), l.T
    return [O, LSE]


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None                                             # whole numbers, and pages copied as they are
    s = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(s)
    return _exact_window(case, s) if case["op"] == "window" else _exact_decode(case, s)
