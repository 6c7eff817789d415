"""64-bit definitions of the serving-step operators: page tables and slots, head
norm with rotation, the 4-bit cache and decode attention over it (numpy, CPU)."""
from __future__ import annotations

import math

import numpy as np
import torch

BK = 128
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def nearest(grid, x):
    """Place in ``grid`` (ascending) of the value nearest to x >= 0; halfway, the even place."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - x, x - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantise(x, gs):
    """(codes [.., D/2] uint8, scales [.., D/16] uint8) of x (float64) [.., D]."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    bad = np.isnan(g).any(-1)
    g = np.where(bad[..., None], 0.0, g)
    amax = np.minimum(np.abs(g).max(-1) / gs, 2688.0)
    sf = nearest(E4M3, amax / 6.0)
    step = E4M3[sf] * gs
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(step[..., None] > 0, np.abs(g) / step[..., None], 0.0)
    code = nearest(GRID, np.minimum(q, 6.0)) + 8 * (np.signbit(g))
    code = code.reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 0x7F, sf).astype(np.uint8)


def values(codes, scales, gs):
    """What codes [.., D/2] and scales [.., D/16] stand for (float64)."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1]).astype(np.int64)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    return v * np.repeat(np.append(E4M3, np.nan)[scales], 16, -1) * gs


def plan(L, n, seq_pt, free, count, N, num_pages):
    """Serial definition of the page-table step; returns a dict and the table."""
    B, mp = seq_pt.shape
    pt, out_len, err = seq_pt.copy(), L.copy(), 0
    slot, pos, seq = (np.full(N, -1, np.int64) for _ in range(3))
    cu, row, off, given = np.zeros(B + 1, np.int64), 0, 0, 0
    top = min(max(count, 0), len(free))
    if top != count:
        err |= 0x10
    for b in range(B):
        cu[b] = min(row, N)
        rows = max(int(n[b]), 0)
        end = int(L[b]) + int(n[b])
        if L[b] < 0 or n[b] < 0 or end > mp * BK or row + rows > N:
            err |= 0x8
            row += rows
            continue
        have, need = -(-int(L[b]) // BK), -(-end // BK) - -(-int(L[b]) // BK)
        if need and off + need > top:
            err |= 0x10
            off += need
            row += rows
            continue
        for i in range(need):
            pt[b, have + i] = free[top - 1 - (off + i)]
        for i in range(rows):
            p = int(L[b]) + i
            page = pt[b, p // BK]
            seq[row + i], pos[row + i] = b, p
            if 0 <= page < num_pages:
                slot[row + i] = int(page) * BK + p % BK
            else:
                err |= 0x2
        out_len[b] = end
        off += need
        given += need
        row += rows
    cu[B] = min(row, N)
    return {"seq_len_out": out_len, "free_count_out": top - given, "cu": cu, "tok_slot": slot, "tok_pos": pos,
            "tok_seq": seq, "seq_pt": pt, "err": err}


def release(L, done, seq_pt, free, count):
    free, out_len, err = free.copy(), L.copy(), 0
    top = min(max(count, 0), len(free))
    if top != count:
        err |= 0x10
    for b in range(len(L)):
        if not done[b]:
            continue
        if L[b] < 0 or L[b] > seq_pt.shape[1] * BK:
            err |= 0x8
            continue
        for j in range(-(-int(L[b]) // BK)):
            if top < len(free):
                free[top] = seq_pt[b, j]
                top += 1
            else:
                err |= 0x10
        out_len[b] = 0
    return {"seq_len_out": out_len, "free_count_out": top, "free_pages": free, "err": err}


def norm_rope(x, weight, pos, inv_freq, eps, interleaved):
    """(y, size) of x [N, H, D]: the definition and the sum of the magnitudes that enter each value."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    size = np.abs(y)
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    if rot:
        t = pos.astype(np.float64)[:, None, None] * inv_freq.astype(np.float64)
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
        u, v, s = a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t), np.abs(a) + np.abs(b)
        y, size = y.copy(), size.copy()
        for z, p, q in ((y, u, v), (size, s, s)):
            if interleaved:
                z[..., 0:rot:2], z[..., 1:rot:2] = p, q
            else:
                z[..., :rot // 2], z[..., rot // 2:rot] = p, q
    return y, size


def attend(q, K, V, scale):
    """(O, LSE, A, Z, S) of q [G, D] over K, V [T, D] (float64): A = sum_t p |v|, Z = max_t scale * sum |q k|,
    S = sum_t |v|."""
    if len(K) == 0:
        return np.zeros_like(q), np.full(len(q), -np.inf), np.zeros_like(q), np.zeros(len(q)), 0.0
    z = q @ K.T * scale
    m = z.max(-1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(-1, keepdims=True)
    p /= l
    Z = (np.abs(q) @ np.abs(K).T).max(-1) * scale
    return p @ V, (m + np.log(l))[:, 0], p @ np.abs(V), Z, np.abs(V).sum(0)


def check_attend(O, LSE, ref):
    """Kernel output of one row against ``attend``'s.

    Scores: 128 exact products summed in fp32 with at most one step (2^-23) lost per
    addition, 128 * 2^-23 of Z at worst, and a few roundings of z and of 2^x (2^-20 of
    1 + Z): dz = 2^-16 (1 + Z).  The probabilities then err by 2 dz, and fp16 rounds
    each by 2^-11; fp32 sums over the tokens add less than 2^-14.  A probability below
    2^-22 of the largest rounds by an absolute amount instead: fp16's subnormal
    steps are 2^-24, half of one 2^-25, and the largest is held as 2^8 at least, so by
    2^-33 of the largest (at most 1) for each token, 2^-33 S in all.  bf16 rounds the result by 2^-8 of it.
    """
    Oe, Le, A, Z, S = ref
    dz = 2.0 ** -16 * (1 + Z)
    lim = 2.0 ** -8 * np.abs(Oe) + (2.0 ** -11 + 2.0 ** -14 + 2 * dz[:, None]) * A + 2.0 ** -33 * S + 1e-30
    bad = ~(np.abs(O - Oe) <= lim)
    assert not bad.any(), f"O off at {np.argwhere(bad)[:3]}, worst {np.nanmax(np.abs(O - Oe) / lim):.3f} of the bound"
    same_inf = np.isneginf(LSE) == np.isneginf(Le)
    assert same_inf.all(), "rows without a token differ"
    on = ~np.isneginf(Le)
    assert (np.abs(LSE[on] - Le[on]) <= dz[on] + 2.0 ** -20 * np.abs(Le[on])).all(), np.abs(LSE[on] - Le[on]).max()


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def default_scale():
    return 1.0 / math.sqrt(128.0)
