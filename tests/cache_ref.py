"""64-bit definitions of the 8-bit cache, window attention with sinks, and shared, moved and freed pages (numpy, CPU)."""
from __future__ import annotations

import math

import numpy as np

BK, D = 128, 128
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])
FIRST, LAST = 87, 167
# half a step of a type, relative to the value: an output's rounding to bf16, and that of P (fp16 over 8-bit pages, else bf16)
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def decode(codes, byte):
    """What codes [..] stand for under scale bytes that broadcast to them."""
    codes = codes.astype(np.int64)
    v = np.append(E4M3, np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    return v * 2.0 ** (np.clip(byte.astype(np.int64), FIRST, LAST) - 127.0)


def encode(x, byte):
    """Codes of x (float64) under scale bytes: nearest, halfway to the even code, past the range to the largest."""
    a = np.abs(x) / 2.0 ** (np.clip(byte.astype(np.int64), FIRST, LAST) - 127.0)
    nan = np.isnan(a)
    a = np.minimum(np.where(nan, 0.0, a), 448.0)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(nan, 127, code + 128 * np.signbit(x)).astype(np.uint8)


def byte_for(amax):
    """The scale byte of a block whose largest finite magnitude is amax."""
    for b in range(FIRST, LAST):
        if amax <= 448 * 2.0 ** (b - 127):
            return b
    return LAST


def store(codes, scales, x, slots):
    """Tokens x [N, H, D] (float64) into codes [P, H, BK, D] and scales [P, H] (both changed in place), one run of rows at a time."""
    N, H, _ = x.shape
    r = 0
    while r < N:
        n = 1
        if slots[r] < 0 or slots[r] // BK >= len(codes):
            r += 1
            continue
        page, t = divmod(int(slots[r]), BK)
        while r + n < N and t + n < BK and slots[r + n] == slots[r] + n:
            n += 1
        for h in range(H):
            new = x[r:r + n, h]
            fin = np.abs(new[np.isfinite(new)])
            byte = byte_for(fin.max() if fin.size else 0.0)
            if t > 0:
                old = min(max(int(scales[page, h]), FIRST), LAST)
                if byte > old:
                    kept = codes[page, h, :t]
                    codes[page, h, :t] = encode(decode(kept, np.array(old)), np.array(byte))
                byte = max(byte, old)
            codes[page, h, t:t + n] = encode(new, np.array(byte))
            scales[page, h] = byte
        r += n


def attend(q, K, V, scale):
    """Of q [G, D] over K, V [T, D]: O [G, D], LSE [G], sum of |p V| / l [G, D] (what errors of P are relative to), the most
    that a token's smallest P may leave out [G, D], and the size of the scores' sums [G]."""
    if len(K) == 0:
        return np.zeros(q.shape), np.full(len(q), -math.inf), np.zeros(q.shape), np.zeros(q.shape), np.zeros(len(q))
    z = q @ K.T * scale
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(1, keepdims=True)
    size = (np.abs(q) @ np.abs(K).T).max(1) * scale
    return p @ V / l, (m + np.log(l))[:, 0], p @ np.abs(V) / l, np.full(q.shape, len(K) * 2.0 ** -31 * np.abs(V).max()), size


def seen(i, window, sinks):
    """The tokens that the query at position i sees."""
    if window == 0:
        return np.arange(i + 1)
    t = np.arange(i + 1)
    return t[(t > i - window) | (t < sinks)]


def check(O, LSE, want, half):
    """O within its own rounding to bf16 and that of each P (`half`: half a step of P's type, and 2^-25 of 2^8 where fp16 ends).
    fp32 scores (128 products, in any order, and two products with scales) are off by less than 2^-19 of their terms'
    size, exponentials and sums by less than 2^-17 together.  LSE: the scores' error, and an fp32 logarithm's and sum's."""
    o, lse, size, least, scores = want
    near = scores[:, None] * 2.0 ** -19 + 2.0 ** -17
    tol = (HALF["bf16"] * np.abs(o) + (half + near) * size) * (1 + 2.0 ** -7) + least + 1e-30
    bad = ~(np.abs(O - o) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], O[bad][:4], o[bad][:4], tol[bad][:4])
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(LSE), empty)
    some = ~empty
    assert np.all(np.abs(LSE[some] - lse[some]) <= near[some, 0] + 2.0 ** -22 * np.abs(lse[some]))


def fork(src, dst, L, pt, free, count, shares):
    """Serial definition of msa_fork_requests."""
    B, mp = pt.shape
    P = len(shares)
    L0, pt, shares, err = L.copy(), pt.copy(), shares.copy(), 0
    L = L.copy()
    top = min(max(count, 0), len(free))
    if top != count:
        err |= 0x10
    copies, named, given, full = [], set(), 0, False
    for s, d in zip(src, dst):
        copies.append((-1, -1))
        if s < 0:
            continue
        if s >= B or not 0 <= d < B or L0[d] != 0:
            err |= 0x20
            continue
        n = int(L0[s])
        if n < 0 or n > mp * BK:
            err |= 0x8
            continue
        if d in named:
            err |= 0x20
            continue
        named.add(d)
        if n % BK:
            if full or given == top:
                full, err = True, err | 0x10
                continue
            page = int(free[top - 1 - given])
            given += 1
            copies[-1] = (int(pt[s, n // BK]), page)
            pt[d, n // BK] = page
        for j in range(n // BK):
            page = pt[s, j]
            pt[d, j] = page
            if 0 <= page < P:
                shares[page] += 1
            else:
                err |= 0x2
        L[d] = n
    c = np.array(copies, dtype=np.int64).reshape(-1, 2)
    return dict(seq_len=L, seq_pt=pt, shares=shares, count=top - given, copy_src=c[:, 0], copy_dst=c[:, 1], err=err)


def release_shared(L, done, pt, free, count, shares):
    """Serial definition of msa_release_shared_pages."""
    L, free, shares, err = L.copy(), free.copy(), shares.copy(), 0
    cap = pt.shape[1] * BK
    top = min(max(count, 0), len(free))
    if top != count:
        err |= 0x10
    for b in range(len(L)):
        if not done[b]:
            continue
        if L[b] < 0 or L[b] > cap:
            err |= 0x8
            continue
        for j in range(-(-int(L[b]) // BK)):
            page = pt[b, j]
            if 0 <= page < len(shares):
                shares[page] -= 1
            else:
                err |= 0x2
        L[b] = 0
    for page in range(len(shares)):
        if shares[page] < 0:
            if shares[page] < -1:
                err |= 0x2
            shares[page] = 0
            if top < len(free):
                free[top] = page
                top += 1
            else:
                err |= 0x10
    return dict(seq_len=L, free=free, count=top, shares=shares, err=err)


def compact(L, pt, shares, cap):
    """Serial definition of msa_compact_pages; the table and counts as outputs of their own."""
    P, err = len(shares), 0
    held = []
    for b in range(len(L)):
        if L[b] < 0 or L[b] > pt.shape[1] * BK:
            err |= 0x8
            continue
        held += [(b, j) for j in range(-(-int(L[b]) // BK))]
    used = {int(pt[b, j]) for b, j in held if 0 <= pt[b, j] < P}
    if any(not 0 <= pt[b, j] < P for b, j in held):
        err |= 0x2
    n = len(used)
    move = list(zip(sorted(p for p in used if p >= n), [p for p in range(n) if p not in used]))
    to = dict(move)
    out, s2 = {}, np.zeros_like(shares)
    for b, j in held:
        out[b, j] = to.get(int(pt[b, j]), int(pt[b, j]))
    for p in used:
        s2[to.get(p, p)] = shares[p]
    free = np.full(cap, -1, np.int64)
    free[:P - n] = P - 1 - np.arange(P - n)
    moves = np.full((P, 2), -1, np.int64)
    if move:
        moves[:len(move)] = move
    return dict(entries=out, shares=s2, free=free, count=P - n, move_src=moves[:, 0], move_dst=moves[:, 1], err=err)
