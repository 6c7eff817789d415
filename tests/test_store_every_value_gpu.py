"""The 4-bit store's kernel over every bf16 value: each finite bit pattern of either sign that a group of a given scale
can hold, beside the value that fixes the scale, against the 64-bit definition."""
import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def bf16(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def groups_of(scale):
    """[n, 16]: largest value 6 scale first (the group's maximum), then every value of at most that size, both signs."""
    every = np.arange(0, 0x7F80, dtype=np.uint32)
    v = bf16(every[bf16(every) <= 6 * scale])
    v = np.concatenate((v, -v))
    v = np.pad(v, (0, -len(v) % 15)).reshape(-1, 15)
    return np.concatenate((np.full((len(v), 1), 6 * scale), v), 1)


def store(msa, x, ks, vs):
    """Codes and scales of x [rows, 128], as keys and as values of one head."""
    N = len(x)
    c = msa.q4_cache(-(-N // 128), 1, "cuda", ks, vs)
    t = torch.from_numpy(x).to(torch.bfloat16).cuda()[:, None]
    assert np.array_equal(ref.f64(t)[:, 0], x)
    msa.msa_cache_append_q4(t, t, torch.arange(N, device="cuda"), c)
    return [a.reshape(-1, a.shape[-1])[:N].cpu().numpy() for a in c[:4]]


def same(codes, scales, x, gs):
    want_codes, want = ref.quantise(x, gs)
    assert np.array_equal(scales, want)
    a, b = (ref.values(k, want, gs) for k in (codes, want_codes))   # -0 and +0 are the same value
    assert np.array_equal(a, b)


@pytest.mark.parametrize("half", range(2))
def test_every_value_under_every_scale(msa, half):
    for places in np.array_split(np.arange(1, 127), 6)[3 * half:3 * half + 3]:
        g = np.concatenate([groups_of(ref.E4M3[i]) for i in places])
        g = np.pad(g, ((0, -len(g) % 8), (0, 0))).reshape(-1, 128)
        Kc, Ks, Vc, Vs = store(msa, g, 1.0, 2.0 ** -3)
        same(Kc, Ks, g, 1.0)
        same(Vc, Vs, g, 2.0 ** -3)


def test_every_value_as_a_groups_largest(msa):
    """Every finite bit pattern alone in its group, under pool scales near and far."""
    every = bf16(np.arange(0, 0x7F80, dtype=np.uint32))
    v = np.concatenate((every, -every))
    g = np.zeros((len(v), 16))
    g[np.arange(len(v)), np.arange(len(v)) % 16] = v
    g = np.pad(g, ((0, -len(g) % 8), (0, 0))).reshape(-1, 128)
    for ks, vs in ((1.0, 2.0 ** -9), (2.0 ** 40, 2.0 ** -40), (2.0 ** 64, 2.0 ** -64)):
        Kc, Ks, Vc, Vs = store(msa, g, ks, vs)
        same(Kc, Ks, g, ks)
        same(Vc, Vs, g, vs)
