"""The serving loop of README.md, run as it stands there: requests that end, sit a step out, are refused for want of
pages and start again, every step against the 64-bit definitions over the tokens each request has been given."""
import math
import os
import re

import numpy as np
import pytest
import torch

import serving_ref as ref
from test_serving_gpu import check_rope, i32, workspace

pytestmark = pytest.mark.gpu
BK = 128
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HQ, HKV, HI, DI = 12, 2, 4, 64


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def readme_blocks():
    """(what is done once, a step) of the serving loop."""
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text[text.index("A serving loop over a 4-bit cache"):], re.S)
    return blocks[0], blocks[1]


class Loop:
    """The names that the README's code uses, and what each request has been given so far."""

    def __init__(self, msa, B, N, max_pages, num_pages, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        f32 = dict(generator=g, device="cuda")
        self.rng, self.fed = np.random.default_rng(seed), [[] for _ in range(B)]
        self.v = v = {
            "msa": msa, "torch": torch, "B": B, "N": N, "Hq": HQ, "Hkv": HKV, "num_pages": num_pages,
            "seq_len": i32(np.zeros(B)), "seq_pt": torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda"),
            "free_pages": torch.randperm(num_pages, **f32).int(), "free_count": i32([num_pages]),
            "new_len": i32(np.zeros(B)), "done": i32(np.zeros(B)),
            "wq": (1 + 0.2 * torch.randn(128, **f32)).bfloat16(), "wk": (1 + 0.2 * torch.randn(128, **f32)).bfloat16(),
            "inv_freq": (5e6 ** (-torch.arange(0, 128, 2, device="cuda").double() / 128)).float(),
            "inv_freq_idx": (5e6 ** (-torch.arange(0, 32, 2, device="cuda").double() / 32)).float(),
            "kidx_pool": torch.zeros(num_pages, HKV, BK, DI, dtype=torch.bfloat16, device="cuda"),
            "O": torch.zeros(B, HQ, 128, dtype=torch.bfloat16, device="cuda"), "LSE": torch.zeros(B, HQ, device="cuda"),
            "ws": workspace(msa, B, HKV)}
        v |= {"Q": torch.zeros(N, HQ, 128, dtype=torch.bfloat16, device="cuda"),
              "q_idx": torch.zeros(N, HKV, HI, DI, dtype=torch.bfloat16, device="cuda"),
              "k_idx": torch.zeros(N, HKV, DI, dtype=torch.bfloat16, device="cuda"), "w": torch.zeros(N, HKV, HI, device="cuda")}
        for x in "KV":
            v[x] = torch.zeros(N, HKV, 128, dtype=torch.bfloat16, device="cuda")
        once, self.code = readme_blocks()
        exec(once, v)
        self.code = compile(self.code, "README.md", "exec")
        self.graph = None

    def capture(self):
        """The step as a graph; its one run without a request changes nothing."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            exec(self.code, self.v)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            exec(self.code, self.v)

    def step(self, new, done):
        v, B, N = self.v, self.v["B"], self.v["N"]
        for x in ("Q", "q_idx", "k_idx", "w", "K", "V"):
            v[x].copy_(torch.from_numpy(self.rng.standard_normal(v[x].shape)).to(v[x].dtype))
        v["new_len"].copy_(i32(new)), v["done"].copy_(i32(done)), v["err"].zero_()
        before = {x: v[x].clone() for x in ("Q", "K", "k_idx")}
        host = lambda x: v[x].cpu().numpy().astype(np.int64)  # noqa: E731
        back = ref.release(host("seq_len"), done, host("seq_pt"), host("free_pages"), int(v["free_count"]))
        want = ref.plan(back["seq_len_out"], np.array(new), host("seq_pt"), back["free_pages"], back["free_count_out"], N, v["num_pages"])
        self.graph.replay() if self.graph else exec(self.code, v)
        torch.cuda.synchronize()
        # tables, norm and rotation
        for x in ("tok_slot", "tok_pos", "tok_seq", "cu"):
            assert np.array_equal(v["plan"][x].cpu(), want[x]), x
        assert np.array_equal(host("seq_len"), want["seq_len_out"]) and int(v["free_count"]) == want["free_count_out"]
        live = torch.from_numpy(want["tok_pos"] >= 0).cuda()
        pos, slot = v["plan"]["tok_pos"][live], v["plan"]["tok_slot"][live]
        check_rope(v["Q"][live], before["Q"][live], v["wq"], pos, v["inv_freq"], False)
        check_rope(v["K"][live], before["K"][live], v["wk"], pos, v["inv_freq"], False)
        check_rope(v["kidx_pool"][slot // BK, :, slot % BK], before["k_idx"][live], None, pos, v["inv_freq_idx"], False)
        assert torch.equal(v["Q"][~live], before["Q"][~live]) and torch.equal(v["K"][~live], before["K"][~live])
        # attention of each request's newest token over all that it has been given (fewer blocks than are selected)
        K, V, Q = ref.f64(v["K"]), ref.f64(v["V"]), ref.f64(v["Q"])
        newest = {}
        for b in range(B):
            if done[b]:
                self.fed[b] = []
            for r in np.flatnonzero(want["tok_seq"] == b):
                self.fed[b].append((K[r], V[r]))
                newest[b] = Q[r]
        assert [len(x) for x in self.fed] == host("seq_len").tolist()
        assert int(v["err"]) == want["err"] | back["err"] and int(v["bufs"]["dev_err"]) == 0
        for O, LSE in ((v["bufs"]["O"], v["bufs"]["LSE"]), (v["O"], v["LSE"])):
            for b in range(B):
                if b not in newest:
                    assert (O[b] == 0).all() and (LSE[b] == -math.inf).all(), b
                    continue
                k, w = (ref.values(*ref.quantise(np.stack([t[i] for t in self.fed[b]]), 1.0), 1.0) for i in (0, 1))
                for g in range(HKV):
                    h = slice(g * HQ // HKV, (g + 1) * HQ // HKV)
                    ref.check_attend(ref.f64(O[b, h]), ref.f64(LSE[b, h]), ref.attend(newest[b][h], k[:, g], w[:, g], ref.default_scale()))
        return newest


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("N", [6, 400])
def test_readme_serving_loop(msa, N, captured):
    B = 6
    loop = Loop(msa, B, N, max_pages=6, num_pages=8, seed=N)
    if captured:
        loop.capture()
    none = [0] * B
    if N > B:
        assert len(loop.step([130, 1, 128, 0, 100, 0], none)) == 4      # prompts: 2 + 1 + 1 + 1 pages of 8
    else:
        assert len(loop.step([1, 1, 1, 0, 3, 0], none)) == 4
    assert set(loop.step([1, 1, 0, 1, 1, 0], none)) == {0, 1, 3, 4}     # request 2 sits out, 3 starts
    assert set(loop.step([1, 0, 1, 0, 1, 1], [0, 1, 0, 0, 0, 0])) == {0, 2, 4, 5}   # request 1 has ended, its page serves another
    if N > B:
        # of 8 pages request 0 has 2, 2 has 2, 3, 4 and 5 one each; request 1 wants two of the one left and is refused,
        # and so are the later ones that need one
        assert set(loop.step([1, 200, 1, 1, 29, 1], none)) == {0, 2, 3, 5}
        assert set(loop.step([1, 100, 0, 1, 29, 1], [0, 0, 1, 0, 0, 0])) == {0, 1, 3, 4, 5}
    assert loop.step(none, [1] * B) == {}                                # all end: a step of empty rows
    assert int(loop.v["free_count"]) == 8
    assert set(loop.step([0, 0, 1, 0, 0, 1], none)) == {2, 5}
