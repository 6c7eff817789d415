"""4-bit decode attention where scores are far outside the range of 2^x: the tokens with the largest score share the
output, whatever its size and sign."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_serving_gpu import check_rows, i32, outputs, q4_pool, workspace

pytestmark = pytest.mark.gpu
BK = 128


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def constant_keys(c, steps):
    """The cache with token t's key steps[page, head, t] (multiples of 1/2 up to 6) in every channel."""
    code = np.searchsorted(ref.GRID, np.abs(steps)) + 8 * (steps < 0)
    codes = np.repeat((code | code << 4).astype(np.uint8)[..., None], 64, -1)
    return c._replace(K_codes=torch.from_numpy(codes).cuda(), K_scales=torch.full_like(c.K_scales, 0x38))   # E4M3: 1


def check_largest(Q, O, LSE, pt, L, c, steps, scale):
    """Equal keys give equal scores, and others lie at least 2^9 apart: the output is the mean of V over the tokens with
    the largest, 2^-11 of each lost to fp16 at most and 2^-14 to the sums, 2^-8 of it to bf16.  The scores' sums are exact,
    the scale and its product round, as does the logarithm's factor: 2^-21 of the log-sum-exp."""
    V = ref.values(c.V_codes.cpu().numpy(), c.V_scales.cpu().numpy(), c.v_scale)
    Hkv, (B, Hq, _), q, o, lse = V.shape[1], Q.shape, ref.f64(Q), ref.f64(O), ref.f64(LSE)
    for b in range(B):
        for h in range(Hq):
            g = h * Hkv // Hq
            pages = [p for p in pt[b] if p >= 0]
            z = np.concatenate([steps[p, g] for p in pages])[:L[b]] * q[b, h, 0] * 128 * scale
            top = z == z.max()
            v = np.concatenate([V[p, g] for p in pages])[:L[b]][top]
            want, size = v.mean(0), np.abs(v).mean(0)
            assert (np.abs(o[b, h] - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14) * size + 1e-30).all()
            assert abs(lse[b, h] - (z.max() + np.log(top.sum()))) <= 2.0 ** -21 * abs(z.max()) + 2.0 ** -16


@pytest.mark.parametrize("power", [4, 18, 20, 22, 23, 24, 25, 26, 27, 28, 30, 40, 63, 90, 110, 117])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(msa, power, sign):
    """Scores of 1.37 * 2^power and more, all of one sign or of both; one token, ties, and a row in many parts."""
    Hkv, P, r = 2, 40, np.random.default_rng(power)
    values = ref.GRID[1:] if power % 2 else np.concatenate((ref.GRID[1:], -ref.GRID[1:]))
    steps = r.choice(values, (P, Hkv, BK))
    c = constant_keys(q4_pool(msa, P, Hkv, 1), steps)
    L = [1, 2, 127, 300, 4000]
    B, Hq = len(L), 8
    per = [-(-x // BK) for x in L]
    ids, at = r.permutation(P), 0
    pt = np.full((B, max(per)), -1)
    for b in range(B):
        pt[b, :per[b]] = ids[at:at + per[b]]
        at += per[b]
    Q = torch.from_numpy(sign * 1.37 * 2.0 ** power / 128 * r.choice([1, 0.75, 1.5], (B, Hq, 1)) * np.ones((B, Hq, 128))).bfloat16().cuda()

    def check(O, LSE, scale):
        if power >= 18:
            check_largest(Q, O, LSE, pt, L, c, steps, scale)
        else:
            check_rows(Q, O, LSE, lambda b, g: pt[b, :per[b]], lambda b, g: L[b], c, scale)
    for scale in (1.0, ref.default_scale()):
        O, LSE = outputs(B, Hq)
        msa.msa_dense_attn_decode_q4(Q, c, i32(pt), i32(L), O, LSE, workspace(msa, B, Hkv), softmax_scale=scale)
        check(O, LSE, scale)
        k = 32
        rows = np.repeat(np.pad(pt, ((0, 0), (0, k - pt.shape[1])), constant_values=-1)[:, :k], Hkv, 0)
        n, last = np.repeat(per, Hkv), np.repeat([x - (p - 1) * BK for x, p in zip(L, per)], Hkv)
        O, LSE = outputs(B, Hq)
        msa.msa_sparse_attn_decode_q4(Q, c, i32(rows), i32(n), i32(last), O, LSE, workspace(msa, B, Hkv), softmax_scale=scale)
        check(O, LSE, scale)
