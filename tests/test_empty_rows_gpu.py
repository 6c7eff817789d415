"""Free rows of a batch (length 0) in the decode step: no tokens, no error, the others as without them."""
import math

import pytest
import torch

from workloads import DecodeWorkload, MSAShape, decode_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as m
    return m


def take(inp, keep):
    return {n: t[keep].contiguous() if n in ("Q", "q_idx", "w", "seq_pt", "seq_len") else t for n, t in inp.items()}


def q4(msa, inp):
    P, Hkv = inp["K_pool"].shape[:2]
    c = msa.q4_cache(P, Hkv, "cuda", 2.0 ** -6, 2.0 ** -6)
    rows = lambda x: x.transpose(1, 2).reshape(P * 128, Hkv, 128)  # noqa: E731
    msa.msa_cache_append_q4(rows(inp["K_pool"]), rows(inp["V_pool"]), torch.arange(P * 128, device="cuda"), c)
    return c


STEPS = {"fused": dict(fused=True), "one_by_one": dict(fused=False)}
CASES = [  # lengths (0: free), k, one index-key pool for all groups
    ((0, 700, 0, 5000, 1, 0), 4, False),
    ((0, 700, 0, 5000, 1, 0), 4, True),
    ((300, 0), 16, False),
    ((0, 270000, 1000), 16, True),          # more than 2048 score blocks: selected after the scores, a block of threads a row
    ((0, 0, 0), 4, False),
]


@pytest.mark.parametrize("lengths,k,shared", CASES)
@pytest.mark.parametrize("form", ["fused", "one_by_one", "q4"])
def test_decode_step_takes_free_rows(msa, lengths, k, shared, form):
    wl = DecodeWorkload("free_rows", lengths=tuple(max(x, 1) for x in lengths), shape=MSAShape(Hq=12, Hkv=2, k=k), seed=91)
    inp = decode_inputs(wl, device="cuda")
    if shared:
        inp["kidx_pool"] = inp["kidx_pool"][:, :1].expand(-1, 2, -1, -1)
    free = torch.tensor([x == 0 for x in lengths], device="cuda")
    inp["seq_len"][free] = 0
    inp["seq_pt"][free] = -1                # as a table row that was never filled
    cache = q4(msa, inp) if form == "q4" else None

    def step(inp, bufs=None, **kw):
        if form == "q4":
            return msa.decode_step_q4(inp, cache, k, bufs=bufs, **kw)
        return msa.decode_step(inp, k, bufs=bufs, **STEPS[form], **kw)

    got = step(inp)
    assert int(got["dev_err"]) == 0
    rows = free.repeat_interleave(2)
    assert (got["O"][free] == 0).all() and (got["LSE"][free] == -math.inf).all() and (got["C"][free] == -math.inf).all()
    assert (got["sel"][free] == -1).all() and (got["count"][free] == 0).all()
    assert (got["pt"][rows] == -1).all() and (got["n"][rows] == 0).all() and (got["last_len"][rows] == 0).all()
    first = {n: got[n].clone() for n in ("O", "LSE", "sel", "n")}
    again = step(inp, got, scratch_zeroed=True)                  # the scratch is left zero
    assert int(again["dev_err"]) == 0 and all(torch.equal(again[n], first[n]) for n in first)
    if not free.all():
        alone = step(take(inp, ~free))
        for n in ("sel", "count"):
            assert torch.equal(alone[n], first.get(n, got[n])[~free]), n
        # (the rows' pages may be cut at other places, so fp32 sums differ in their last bits and bf16 by a step)
        assert torch.allclose(alone["O"].float(), first["O"][~free].float(), rtol=2 ** -7, atol=1e-4)
        assert torch.allclose(alone["LSE"], first["LSE"][~free], rtol=2 ** -16, atol=2 ** -16)


def test_lengths_below_zero_stay_an_error(msa):
    wl = DecodeWorkload("bad_rows", lengths=(700, 300), shape=MSAShape(Hq=12, Hkv=2, k=4), seed=92)
    inp = decode_inputs(wl, device="cuda")
    inp["seq_len"][1] = -1
    for fused in (True, False):
        out = msa.decode_step(inp, 4, fused=fused)
        assert int(out["dev_err"]) == msa.MSA_DEVERR_BAD_LEN
        assert (out["O"][1] == 0).all() and (out["LSE"][1] == -math.inf).all()
