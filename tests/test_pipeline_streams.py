"""Pipelines on a stream of the caller's that allocate their own buffers: on the CPU, where they ask torch for them; on
the GPU, the results beside work that still uses the memory torch gave back on the current stream."""
import contextlib

import pytest
import torch

import block_sparse_attention_02_gb300 as msa


def test_buffers_are_made_on_the_given_stream(monkeypatch):
    inside, made = [], []

    @contextlib.contextmanager
    def stream(s):
        inside.append(s)
        yield
        inside.pop()

    class Stream:
        pass
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p, device: ("external", p))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: "default")
    for name in [n for n in dir(msa) if n.startswith("msa_") and callable(getattr(msa, n))]:
        monkeypatch.setattr(msa, name, lambda *a, **k: 16)
    for name in ("decode_buffers", "decode_q4_buffers", "prefill_buffers", "chunk_buffers", "dense_decode_buffers"):
        def buffers(*a, _real=getattr(msa, name), **k):
            made.append(list(inside))
            return _real(*a, **k)
        monkeypatch.setattr(msa, name, buffers)
    e = torch.empty
    pools = {"K_pool": e(3, 2, 128, 128), "V_pool": e(3, 2, 128, 128), "kidx_pool": e(3, 2, 128, 64), "seq_pt": e(1, 3).int(),
             "seq_len": e(1).int(), "q_pos": e(1).int()}
    step = {"Q": e(1, 4, 128), "q_idx": e(1, 2, 4, 64), "w": e(1, 2, 4), **pools}
    rows = {"Q": e(1, 5, 4, 128), "K": e(1, 5, 2, 128), "V": e(1, 5, 2, 128), "q_idx": e(1, 5, 2, 4, 64), "k_idx": e(1, 5, 2, 64),
            "w": e(1, 5, 2, 4), **pools}
    cache = msa.q4_cache(3, 2, "cpu")
    s = Stream()
    for given, want in ((s, [s]), (1234, [("external", 1234)]), (0, ["default"]), (None, [])):
        for call in (lambda: msa.decode_step(step, 2, stream=given), lambda: msa.decode_step_q4(step, cache, 2, stream=given),
                     lambda: msa.prefill_layer(rows, 2, stream=given), lambda: msa.chunk_layer(rows, 2, stream=given),
                     lambda: msa.dense_decode_step(step, stream=given)):
            made.clear()
            call()
            assert made and all(m == want for m in made), (given, made)
            assert inside == []


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("form", ["bf16", "q4"])
def test_step_on_a_side_stream_beside_unfinished_work(form, raw):
    """The current stream sleeps, then fills memory that torch has been given back: the step's buffers are not in it."""
    import __graft_entry__ as g
    g.build()
    from workloads import DecodeWorkload, MSAShape, decode_inputs
    wl = DecodeWorkload("side", lengths=(700, 5000, 300), shape=MSAShape(Hq=12, Hkv=2, k=4), seed=93)
    inp = decode_inputs(wl, device="cuda")
    P = inp["K_pool"].shape[0]
    cache = msa.q4_cache(P, 2, "cuda", 2.0 ** -6, 2.0 ** -6)
    rows = lambda x: x.transpose(1, 2).reshape(P * 128, 2, 128)  # noqa: E731
    msa.msa_cache_append_q4(rows(inp["K_pool"]), rows(inp["V_pool"]), torch.arange(P * 128, device="cuda"), cache)

    def step(stream=None):
        return msa.decode_step_q4(inp, cache, 4, stream=stream) if form == "q4" else msa.decode_step(inp, 4, stream=stream)
    want = {n: step()[n].clone() for n in ("O", "LSE", "sel")}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    back = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in [512] * 20 + [20000] * 10 + [1 << 21] * 4 + [12 << 20] * 2]
    for t in back:
        t.fill_(0x11)
    del back, t
    got = step(side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert int(got["dev_err"]) == 0
    for n in want:
        assert torch.equal(got[n], want[n]), n
