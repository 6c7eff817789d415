"""Requests that are shortened, as rejected draft tokens do: within their last page by the length alone, into pages that others hold by a
fork at the lower length and the old row's release."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from test_cache_q8_gpu import tokens

pytestmark = pytest.mark.gpu
BK, D, H, P, MOST = 128, 128, 2, 16, 4


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Four rows over one cache, with what each of them should hold."""

    def __init__(self, msa):
        self.msa, self.g = msa, torch.Generator().manual_seed(3)
        self.cache = msa.q8_cache(P, H, "cuda")
        self.L, self.pt = i32([0] * 4), torch.full((4, MOST), -1, dtype=torch.int32, device="cuda")
        self.free, self.n, self.shares, self.e = torch.randperm(P, device="cuda").int(), i32([P]), i32([0] * P), i32([0])

    def append(self, row, n, size=1.0):
        new = [0] * 4
        new[row] = n
        plan = self.msa.plan_buffers(4, n, "cuda")
        self.msa.msa_plan_step(self.L, i32(new), self.pt, self.free, self.n, self.L, self.n, plan["cu"], plan["tok_slot"], plan["tok_pos"],
                               plan["tok_seq"], num_pages=P, dev_err=self.e)
        K, V = tokens(self.g, n, H, size)
        self.msa.msa_cache_append_q8(K.cuda(), V.cuda(), plan["tok_slot"], self.cache, dev_err=self.e)
        return K, V

    def fork(self, src, dst, L=None):
        """From L tokens of src (all of them if not given)."""
        cut, out, c = self.L.clone(), self.L.clone(), (i32([0]), i32([0]))
        if L is not None:
            cut[src] = L
        self.msa.msa_fork_requests(i32([src]), i32([dst]), cut, self.pt, self.free, self.n, self.shares, out, self.pt, self.n, self.shares,
                                   *c, dev_err=self.e)
        self.msa.msa_copy_pages(list(self.cache), *c, dev_err=self.e)
        self.L[dst] = out[dst]

    def release(self, row):
        done = [0] * 4
        done[row] = 1
        self.msa.msa_release_shared_pages(self.L, i32(done), self.pt, self.free, self.n, self.shares, self.L, self.n, self.shares,
                                          dev_err=self.e)

    def values(self, row):
        """K of the row's tokens [L, H, D]."""
        L = int(self.L[row])
        t = torch.arange(L, device="cuda")
        page = self.pt[row].long()[t // BK]
        codes, scales = self.cache.K_codes[page, :, t % BK].cpu().numpy(), self.cache.K_scales[page].cpu().numpy()
        return ref.decode(codes, scales[..., None])

    def check(self):
        """No error; every page is on the stack or held, and counted as often as it is held beyond once."""
        assert int(self.e) == 0
        L, pt, n = self.L.cpu().numpy(), self.pt.cpu().numpy(), int(self.n)
        held = np.concatenate([pt[b, :-(-int(L[b]) // BK)] for b in range(4)]) if L.any() else np.zeros(0, int)
        free = self.free.cpu().numpy()[:n]
        times = np.bincount(held, minlength=P)
        assert np.array_equal(np.sort(free), np.flatnonzero(times == 0))
        assert np.array_equal(self.shares.cpu().numpy(), np.maximum(times - 1, 0))


@pytest.mark.parametrize("lower", [1, 128, 200, 256, 299])
def test_into_shared_pages(msa, lower):
    s = Server(msa)
    s.append(0, 300)
    s.fork(0, 1)                                  # two full pages are both rows', the third one has a copy
    s.append(1, 10)
    other, own = s.values(1), s.values(0)
    s.fork(0, 2, lower)
    s.release(0)
    s.check()
    assert int(s.L[2]) == lower and np.array_equal(s.values(2), own[:lower])
    s.append(2, 150, size=50.0)
    s.check()
    assert np.array_equal(s.values(1), other)
    if lower % BK == 0:                           # (else the page's scale has grown: values may have been rounded again)
        assert np.array_equal(s.values(2)[:lower], own[:lower])
    for row in (1, 2):
        s.release(row)
    s.check()
    assert int(s.n) == P


def test_within_the_last_page(msa):
    """The dropped tokens' scale stays, the values are right to its step; another row's pages are as they were."""
    s = Server(msa)
    K0, _ = s.append(0, 140)
    s.fork(0, 1)
    other = s.values(1)
    s.append(0, 4, size=1000.0)                   # drafts, far larger
    scale = s.cache.K_scales[s.pt[0, 1].long()].cpu().numpy().copy()
    s.L[0] = 140
    K1, _ = s.append(0, 5)
    s.check()
    assert np.array_equal(s.cache.K_scales[s.pt[0, 1].long()].cpu().numpy(), scale)
    want = torch.cat([K0, K1]).double().numpy()
    # 2^-4 of a value, twice where it was rounded again, and half a subnormal step (2^-10) of the block's scale each time
    step = np.concatenate([ref.decode(np.full((128, H, 1), 0x38, np.uint8), s.cache.K_scales[s.pt[0, 0].long()].cpu().numpy()[None, :, None]),
                           np.broadcast_to(2.0 ** (scale.astype(float) - 127)[None, :, None], (17, H, 1))])
    assert np.all(np.abs(s.values(0) - want) <= 2 * (np.abs(want) * 2.0 ** -4 + step * 2.0 ** -10) * (1 + 2.0 ** -4))
    assert np.array_equal(s.values(1), other)
