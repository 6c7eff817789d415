"""Rotation by frequencies of any size: the angle against exact integer arithmetic, and frequencies that are not finite."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref
from test_serving_gpu import rope_case

pytestmark = pytest.mark.gpu
BITS = 512


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def turn():
    """1 / (2 pi) in units of 2^-BITS (Machin's formula)."""
    one = 1 << (2 * BITS)

    def arctan_of_inverse(n):
        term, total, k, sign = one // n, 0, 1, 1
        while term:
            total += sign * (term // k)
            term //= n * n
            k, sign = k + 2, -sign
        return total
    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    return (one << BITS) // (2 * pi)


def angles(pos, f):
    """pos * f modulo 2 pi in radians, [N, len(f)]; every f a whole number."""
    inv = turn()
    out = [[((p * int(v) * inv) % (1 << BITS)) / (1 << BITS) for v in f] for p in pos]
    return 2 * math.pi * np.array(out)


def rotated(x, t):
    """(y, size) of x [N, H, 128] turned by t [N, 64] in split pairs."""
    a, b, t = x[..., :64], x[..., 64:], t[:, None]
    y = np.concatenate((a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)), -1)
    return y, np.tile(np.abs(a) + np.abs(b), 2)


def test_norm_rope_large_frequencies(msa):
    """Whole frequencies from 2^22 to the largest float, positions to 2^20."""
    Q, _, _, _, _, pos, _ = rope_case(70, 3, 1, 128, 128, 21, far=1 << 20)
    r = np.random.default_rng(5)
    f = (np.floor(2.0 ** r.uniform(22, 127.9, 64)) * r.choice([-1, 1], 64)).astype(np.float32)
    f[:12] = [2.0 ** 23, 2.0 ** 24, -2.0 ** 24, 2.0 ** 24 + 2, 2.0 ** 31, 2.0 ** 55, 2.0 ** 56, 1e10, 1e20, -1e30, np.finfo(np.float32).max, -2.0 ** 127]
    pos[:3] = torch.tensor([0, 1, (1 << 20) - 1])
    Qo = torch.empty_like(Q)
    msa.msa_qk_norm_rope(Q, None, pos, torch.from_numpy(f).cuda(), Qo, None)
    y, size = rotated(ref.f64(Q), angles(pos.tolist(), f.tolist()))
    # the sines' 2^-21 and the angle's fp32 fraction of a half turn, 2^-24 of at most pi, then bf16's 2^-8
    assert (np.abs(ref.f64(Qo) - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -16 * size + 1e-30).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_frequencies_that_are_not_finite(msa, interleaved):
    """Exactly the pairs of such a frequency are NaN, at position 0 too."""
    N = 20
    Q, K, _, wq, _, pos, f = rope_case(N, 3, 2, 128, 128, 22)
    pos[4] = 0
    bad = [0, 5, 31, 32, 63]
    f[bad] = torch.tensor([math.inf, -math.inf, math.nan, math.inf, math.nan], device="cuda")
    Qo, Ko = torch.empty_like(Q), torch.empty_like(K)
    msa.msa_qk_norm_rope(Q, K, pos, f, Qo, Ko, q_weight=wq, interleaved=interleaved)
    hit = torch.zeros(128, dtype=torch.bool, device="cuda")
    for i in bad:
        hit[[2 * i, 2 * i + 1] if interleaved else [i, i + 64]] = True
    for o in (Qo, Ko):
        assert torch.isnan(o[..., hit]).all() and torch.isfinite(o[..., ~hit]).all()
    clean = f.clone()
    clean[bad] = 1.0
    Qc, Kc = torch.empty_like(Q), torch.empty_like(K)
    msa.msa_qk_norm_rope(Q, K, pos, clean, Qc, Kc, q_weight=wq, interleaved=interleaved)
    assert torch.equal(Qo[..., ~hit], Qc[..., ~hit]) and torch.equal(Ko[..., ~hit], Kc[..., ~hit])
