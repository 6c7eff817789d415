"""A chunk's layer over a prefix held in 4 bits: the sequences' pages expanded into pools of their own, with their own
page table, beside index keys in the cache's pages."""
import math

import numpy as np
import pytest
import torch

import oracle
from msa_check import check_attention
from workloads import ChunkWorkload, MSAShape, chunk_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


@pytest.mark.parametrize("wl", [ChunkWorkload("q4_chunk", prefix=(300, 1000), S=200, shape=MSAShape(Hq=12, Hkv=2, k=4), seed=71),
                                ChunkWorkload("q4_verify", prefix=(1000, 129, 4000, 60), S=4, shape=MSAShape(Hq=12, Hkv=2, k=4), seed=72)],
                         ids=["chunk", "verify"])
def test_chunk_over_expanded_pages(msa, wl):
    inp, sh = chunk_inputs(wl, device="cuda"), wl.shape
    P, Bk = inp["K_pool"].shape[0], sh.Bk
    # the cache: twice the pages, the sequences' ones spread over it, the index keys in the same pages
    place = torch.randperm(2 * P, generator=torch.Generator().manual_seed(1)).cuda()[:P]
    cache = msa.q4_cache(2 * P, sh.Hkv, "cuda", 2.0 ** -6, 2.0 ** -6)
    rows = lambda x: x.transpose(1, 2).reshape(P * Bk, sh.Hkv, 128)  # noqa: E731
    slots = (place[:, None] * Bk + torch.arange(Bk, device="cuda")).flatten()
    msa.msa_cache_append_q4(rows(inp["K_pool"]), rows(inp["V_pool"]), slots, cache)
    kidx = torch.zeros(2 * P, *inp["kidx_pool"].shape[1:], dtype=torch.bfloat16, device="cuda")
    kidx[place] = inp["kidx_pool"]
    table = torch.where(inp["seq_pt"] >= 0, place[inp["seq_pt"].clamp(min=0).long()].int(), -1)
    # the sequences' pages, one after another, and their table
    per = [(p + wl.S + Bk - 1) // Bk for p in wl.prefix]
    pages = torch.cat([table[b, :n] for b, n in enumerate(per)])
    own = torch.full_like(table, -1)
    for b, n in enumerate(per):
        own[b, :n] = sum(per[:b]) + torch.arange(n, dtype=torch.int32, device="cuda")
    Kx, Vx = (torch.empty(len(pages), sh.Hkv, Bk, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    msa.msa_cache_expand_q4(cache, pages, Kx, Vx)
    got = msa.chunk_layer({**{n: inp[n] for n in ("Q", "q_idx", "w", "q_pos")}, "K_pool": Kx, "V_pool": Vx, "kidx_pool": kidx,
                           "seq_pt": table.contiguous(), "kv_seq_pt": own.contiguous()}, sh.k)
    plain = msa.chunk_layer(inp, sh.k)
    assert int(got["dev_err"]) == 0 and int(plain["dev_err"]) == 0
    for n in ("C", "sel", "count"):                              # the index branch does not see the cache's values
        assert torch.equal(got[n], plain[n]), n
    O, LSE = oracle.chunk_attend(inp["Q"].cpu(), Kx.cpu(), Vx.cpu(), own.cpu(), inp["q_pos"].cpu(), got["sel"].cpu().numpy(),
                                 got["count"].cpu().numpy(), 1.0 / math.sqrt(sh.D), Bk)
    check_attention(got["O"].float().cpu().numpy(), got["LSE"].cpu().numpy(), O, LSE)
    # expanded are the cache's values of these pages, whatever their order
    back = torch.randperm(len(pages)).cuda()
    K2, V2 = torch.empty_like(Kx), torch.empty_like(Vx)
    msa.msa_cache_expand_q4(cache, pages[back].contiguous(), K2, V2)
    assert torch.equal(K2, Kx[back]) and torch.equal(V2, Vx[back]) and np.isfinite(LSE).all()
