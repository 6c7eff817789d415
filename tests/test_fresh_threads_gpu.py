"""Calls that describe tensors to the copy engine, from a thread that has not used the GPU yet: as from the main thread."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
BK, D = 128, 128


def calls(msa):
    """{name: (f(stream), outputs)}"""
    from workloads import ChunkWorkload, DecodeWorkload, MSAShape, PrefillWorkload, chunk_inputs, decode_inputs, prefill_inputs
    sh = MSAShape(Hq=12, Hkv=2, k=4)
    dec = decode_inputs(DecodeWorkload("threads", lengths=(700, 3000), shape=sh, seed=5), device="cuda:0")
    pre = prefill_inputs(PrefillWorkload("threads", B=1, S=700, shape=sh, seed=6), device="cuda:0")
    chunk = chunk_inputs(ChunkWorkload("threads", prefix=(500, 900), S=40, shape=sh, seed=7), device="cuda:0")
    out = {}

    def add(name, f):
        bufs = f(None, None)
        torch.cuda.synchronize()
        out[name] = (lambda s, f=f, b=bufs: f(b, s), {n: bufs[n] for n in ("O", "LSE")})

    add("decode step", lambda b, s: msa.decode_step(dec, 4, b, stream=s))
    add("decode step, calls apart", lambda b, s: msa.decode_step(dec, 4, b, stream=s, fused=False))
    add("dense decode", lambda b, s: msa.dense_decode_step(dec, b, stream=s))
    add("prefill", lambda b, s: msa.prefill_layer(pre, 4, b, stream=s))
    add("dense prefill", lambda b, s: msa.dense_prefill_layer(pre, b, stream=s))
    add("chunk", lambda b, s: msa.chunk_layer(chunk, 4, b, stream=s))

    def window(inp, **kw):
        def f(b, s):
            b = b or {"O": torch.empty_like(inp["Q"]), "LSE": torch.empty(inp["Q"].shape[:3], device="cuda")}
            msa.msa_window_attn_prefill(inp["Q"], inp.get("K", inp.get("K_pool")), inp.get("V", inp.get("V_pool")), b["O"], b["LSE"],
                                        window=200, sinks=4, stream=s, **kw)
            return b
        return f
    add("window prefill", window(pre))
    add("window prefill over pages", window(chunk, seq_pt=chunk["seq_pt"], q_pos=chunk["q_pos"]))
    return out


@pytest.mark.parametrize("given", [False, True])
def test_first_call_of_a_thread(given):
    import __graft_entry__ as g
    g.build()
    import block_sparse_attention_02_gb300 as msa
    stream = torch.cuda.Stream()
    for name, (f, out) in calls(msa).items():
        want = {n: t.clone() for n, t in out.items()}
        for t in out.values():
            t.zero_()
        torch.cuda.synchronize()
        wrong = []

        def work():
            try:
                f(stream if given else None)
            except Exception as e:       # noqa: BLE001 (a thread's own exception would not fail the test)
                wrong.append(str(e))
        thread = threading.Thread(target=work)
        thread.start()
        thread.join()
        torch.cuda.synchronize()
        assert not wrong, (name, wrong)
        for n, t in out.items():
            assert torch.equal(t, want[n]), (name, n)
