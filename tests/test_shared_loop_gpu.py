"""README.md's loop over an 8-bit cache with forks, run as it stands there, eager and captured: a forked request answers as
its source does, and each one's window attention is that of its own tokens."""
import os
import re

import numpy as np
import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu
BK, D, HQ, HKV, HI, DI = 128, 128, 12, 2, 4, 64
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def readme_blocks():
    text = open(os.path.join(ROOT, "README.md")).read()
    return re.findall(r"```python\n(.*?)```", text[text.index("Over an 8-bit cache, with requests"):], re.S)[:2]


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("captured", [False, True])
def test_readme_loop_with_forks(captured):
    import __graft_entry__ as entry
    entry.build()
    import block_sparse_attention_02_gb300 as msa
    B, N, P, most = 4, 300, 12, 6
    g = torch.Generator(device="cuda").manual_seed(31)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    v = {"msa": msa, "torch": torch, "B": B, "N": N, "Hq": HQ, "Hkv": HKV, "num_pages": P,
         "seq_len": i32([0] * B), "seq_pt": torch.full((B, most), -1, dtype=torch.int32, device="cuda"),
         "free_pages": torch.randperm(P, generator=g, device="cuda").int(), "free_count": i32([P]), "new_len": i32([0] * B),
         "done": i32([0] * B), "src": i32([-1, -1]), "dst": i32([-1, -1]), "copy_src": i32([-1, -1]), "copy_dst": i32([-1, -1]),
         "inv_freq": (1e4 ** (-torch.arange(0, 128, 2, device="cuda").double() / 128)).float(),
         "inv_freq_idx": (1e4 ** (-torch.arange(0, 32, 2, device="cuda").double() / 32)).float(),
         "kidx_pool": torch.zeros(P, HKV, BK, DI, dtype=torch.bfloat16, device="cuda"),
         "O": torch.zeros(B, HQ, D, dtype=torch.bfloat16, device="cuda"), "LSE": torch.zeros(B, HQ, device="cuda")}
    sizes = {"Q": (N, HQ, D), "K": (N, HKV, D), "V": (N, HKV, D), "q_idx": (N, HKV, HI, DI), "k_idx": (N, HKV, DI)}
    v |= {n: rand(*s) for n, s in sizes.items()} | {"w": torch.rand(N, HKV, HI, generator=g, device="cuda")}
    once, code = readme_blocks()
    exec(once, v)
    code = compile(code, "README.md", "exec")
    graph = None
    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            exec(code, v)                                    # (no request: it changes nothing)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            exec(code, v)

    def step(new, done=(0, 0, 0, 0), src=(-1, -1), dst=(-1, -1), same=()):
        for n, s in sizes.items():
            v[n].copy_(rand(*s))
        for a, b in same:                                    # token row a as row b
            for n in (*sizes, "w"):
                v[n][a] = v[n][b]
        for n, x in (("new_len", new), ("done", done), ("src", src), ("dst", dst)):
            v[n].copy_(i32(x))
        graph.replay() if graph else exec(code, v)
        torch.cuda.synchronize()
        assert int(v["err"].item()) == 0 and int(v["bufs"]["dev_err"].item()) == 0
        K, V = (torch.empty(P, HKV, BK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        msa.msa_cache_expand_q8(v["cache"], torch.arange(P, dtype=torch.int32, device="cuda"), K, V)
        k, w, q, pt = host(K), host(V), host(v["step"]["Q"]), v["seq_pt"].cpu().numpy()
        for b, L in enumerate(v["step"]["seq_len"].tolist()):
            t = np.arange(L)
            for h in range(HKV):
                at = slice(h * HQ // HKV, (h + 1) * HQ // HKV)
                for O, LSE in ((v["O"], v["LSE"]), (v["bufs"]["O"], v["bufs"]["LSE"])):   # (fewer pages than are selected)
                    ref.check(host(O[b, at]), LSE[b, at].double().cpu().numpy(),
                              ref.attend(q[b, at], k[pt[b, t // BK], h, t % BK], w[pt[b, t // BK], h, t % BK], D ** -0.5), ref.HALF["fp16"])
        return [(v[n] if n in v else v["bufs"][n]).clone() for n in ("O", "LSE")] + [v["bufs"]["O"].clone()]

    step([200, 5, 0, 0])
    assert v["seq_len"].tolist() == [200, 5, 0, 0] and int(v["free_count"]) == P - 3
    # request 2 goes on from request 0, request 3 from request 1 (a page that is partly filled, and no full one)
    got = step([1, 1, 1, 1], src=(0, 1), dst=(2, 3), same=[(2, 0), (3, 1)])
    assert v["seq_len"].tolist() == [201, 6, 201, 6] and int(v["free_count"]) == P - 5 and v["shares"].sum() == 1
    for x in got:
        assert torch.equal(x[0], x[2]) and torch.equal(x[1], x[3])
    # they part; then the sources end, and what they shared stays with the others
    got = step([1, 1, 1, 1])
    assert not torch.equal(got[0][0], got[0][2])
    step([0, 0, 60, 125], done=(1, 1, 0, 0))
    assert v["seq_len"].tolist() == [0, 0, 262, 132] and v["shares"].sum() == 0 and int(v["free_count"]) == P - 5
    step([0, 0, 0, 0], done=(0, 0, 1, 1))
    assert int(v["free_count"]) == P and sorted(v["free_pages"].tolist()) == list(range(P))
