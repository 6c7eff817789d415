"""decode_step_q4 with tensors on another device than the current one: both of its calls are made with theirs current."""
import contextlib
import types

import torch

import block_sparse_attention_02_gb300 as msa


def test_decode_step_q4_runs_on_its_tensors_device(monkeypatch):
    current, calls = [0], []

    @contextlib.contextmanager
    def device(d):
        old, current[0] = current[0], d.index
        yield
        current[0] = old
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    for name in ("msa_index_score", "msa_sparse_attn_decode_q4"):
        monkeypatch.setattr(msa, name, lambda *a, _n=name, **k: calls.append((_n, current[0], k.get("scratch_zeroed"))))
    bufs = dict.fromkeys(("dev_err", "C", "sel", "count", "pt", "n", "last_len", "row_scratch", "O", "LSE", "ws"))
    cache = msa.q4_cache(2, 2, "cpu")
    for index in (0, 1):
        Q = types.SimpleNamespace(shape=(3, 4, 128), device=torch.device("cuda", index))
        inp = dict.fromkeys(("q_idx", "w", "kidx_pool", "seq_pt", "seq_len"), None) | {"Q": Q}
        calls.clear()
        assert msa.decode_step_q4(inp, cache, 16, bufs=bufs, scratch_zeroed=True) is bufs
        assert calls == [("msa_index_score", index, True), ("msa_sparse_attn_decode_q4", index, True)]
        assert current == [0]
