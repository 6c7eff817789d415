"""Refusals of the 8-bit cache, window attention and shared-page entry points without a GPU: struct layouts, argument
checks of the C calls (nothing is enqueued) and of the Python wrappers."""
import ctypes as C
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: every call below fails validation first
INV, UNS, WS = 1, 2, 5


@pytest.fixture(scope="module")
def abi():
    from block_sparse_attention_02_gb300 import build as b
    b.build()
    from block_sparse_attention_02_gb300 import _abi
    _abi.load()
    return _abi


def test_struct_layout_matches_header(abi, tmp_path):
    structs = {"msa_q8_cache": abi.Q8CacheArgs, "msa_append_q8_args": abi.AppendQ8Args, "msa_expand_q8_args": abi.ExpandQ8Args,
               "msa_decode_q8_args": abi.DecodeQ8Args, "msa_dense_decode_q8_args": abi.DenseDecodeQ8Args,
               "msa_window_decode_args": abi.WindowDecodeArgs, "msa_window_prefill_args": abi.WindowPrefillArgs,
               "msa_fork_args": abi.ForkArgs, "msa_release_shared_args": abi.ReleaseSharedArgs, "msa_compact_args": abi.CompactArgs,
               "msa_copy_pages_args": abi.CopyPagesArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "msa.h"', "int main(void) {",
             'printf("consts %d %d\\n", MSA_MAX_POOLS, MSA_DEVERR_BAD_ROW);']
    for c, py in structs.items():
        lines.append(f'printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    out = subprocess.check_output([str(exe)], text=True).splitlines()
    assert out[0] == f"consts {abi.MSA_MAX_POOLS} {abi.MSA_DEVERR_BAD_ROW}"
    for line in out[1:]:
        s, f, v = line.split()
        assert int(v) == (C.sizeof(structs[s]) if f == "size" else getattr(structs[s], f).offset), line


def make(cls, **kw):
    """A struct with every pointer set, and the given fields."""
    a = cls()
    for f, t in cls._fields_:
        if t is C.c_void_p and f != "dev_err":
            setattr(a, f, FAKE)
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(a, k)[:len(v)] = v
        else:
            setattr(a, k, v)
    return a


def q8(abi, **kw):
    return make(abi.Q8CacheArgs, **{**dict(code_stride=(32768, 16384), scale_stride=(2, 1), num_pages=9), **kw})


def append_args(abi, cache=None, **kw):
    return make(abi.AppendQ8Args, **{**dict(N=4, Hkv=2, D=128, Bk=128, K_stride=(256, 128), V_stride=(256, 128)), **kw,
                                     "cache": cache or q8(abi)})


def expand_args(abi, cache=None, **kw):
    return make(abi.ExpandQ8Args, **{**dict(n=4, Hkv=2, D=128, Bk=128), **kw, "cache": cache or q8(abi)})


def sparse_args(abi, cache=None, **kw):
    return make(abi.DecodeQ8Args, **{**dict(B=2, Hq=12, Hkv=2, D=128, Bk=128, k=16, Q_stride=(1536, 128)), **kw,
                                     "cache": cache or q8(abi)})


def dense_args(abi, cache=None, **kw):
    return make(abi.DenseDecodeQ8Args, **{**dict(B=2, Hq=12, Hkv=2, D=128, Bk=128, Q_stride=(1536, 128), max_pages=8), **kw,
                                          "cache": cache or q8(abi)})


def window_args(abi, **kw):
    return make(abi.WindowDecodeArgs, **{**dict(B=2, Hq=12, Hkv=2, D=128, Bk=128, Q_stride=(1536, 128), kv_stride=(32768, 16384, 128),
                                                num_pages=9, max_pages=8, window=64, sinks=4), **kw})


def prefill_args(abi, **kw):
    return make(abi.WindowPrefillArgs, **{**dict(
        mode=0, B=2, S=40, Hq=12, Hkv=2, D=128, Bk=128, window=64, sinks=4, Q_stride=(61440, 1536, 128), K_stride=(10240, 256, 128),
        V_stride=(10240, 256, 128)), **kw})


def chunk_args(abi, **kw):
    return prefill_args(abi, **{**dict(mode=2, K_stride=(32768, 16384, 128), V_stride=(32768, 16384, 128), num_pages=9, max_pages=8), **kw})


def fork_args(abi, **kw):
    return make(abi.ForkArgs, **{**dict(B=4, F=3, Bk=128, max_pages=8, free_cap=32, num_pages=32), **kw})


def release_args(abi, **kw):
    return make(abi.ReleaseSharedArgs, **{**dict(B=4, Bk=128, max_pages=8, free_cap=32, num_pages=32), **kw})


def compact_args(abi, **kw):
    return make(abi.CompactArgs, **{**dict(B=4, Bk=128, max_pages=8, free_cap=32, num_pages=32), **kw})


def copy_args(abi, **kw):
    return make(abi.CopyPagesArgs, **{**dict(n=4, num_pages=9, pools=2, pool=(FAKE, FAKE), page_stride=(512, 300), page_bytes=(512, 17)), **kw})


REFUSED = [
    ("msa_cache_append_q8", append_args, dict(D=64), UNS), ("msa_cache_append_q8", append_args, dict(Bk=64), UNS),
    ("msa_cache_append_q8", append_args, dict(N=-1), INV), ("msa_cache_append_q8", append_args, dict(N=1 << 31), INV),
    ("msa_cache_append_q8", append_args, dict(Hkv=0), INV), ("msa_cache_append_q8", append_args, dict(slots=None), INV),
    ("msa_cache_append_q8", append_args, dict(V_stride=(256, 4)), INV), ("msa_cache_append_q8", append_args, dict(K_stride=(0, 128)), INV),
    ("msa_cache_append_q8", append_args, dict(K=FAKE + 2), INV),
    ("msa_cache_expand_q8", expand_args, dict(n=-1), INV), ("msa_cache_expand_q8", expand_args, dict(pages=None), INV),
    ("msa_cache_expand_q8", expand_args, dict(V_out=FAKE + 8), INV),
    ("msa_sparse_attn_decode_q8", sparse_args, dict(B=4097), INV), ("msa_sparse_attn_decode_q8", sparse_args, dict(k=65), UNS),
    ("msa_sparse_attn_decode_q8", sparse_args, dict(k=0), UNS), ("msa_sparse_attn_decode_q8", sparse_args, dict(Hq=18), UNS),
    ("msa_sparse_attn_decode_q8", sparse_args, dict(Hq=13), UNS), ("msa_sparse_attn_decode_q8", sparse_args, dict(D=64), UNS),
    ("msa_sparse_attn_decode_q8", sparse_args, dict(B=4096, Hq=1 << 15, Hkv=1 << 13), UNS),
    ("msa_sparse_attn_decode_q8", sparse_args, dict(pt=None), INV), ("msa_sparse_attn_decode_q8", sparse_args, dict(O=None), INV),
    ("msa_sparse_attn_decode_q8", sparse_args, dict(Q_stride=(1536, 100)), INV),
    ("msa_dense_attn_decode_q8", dense_args, dict(B=1025), INV), ("msa_dense_attn_decode_q8", dense_args, dict(max_pages=0), INV),
    ("msa_dense_attn_decode_q8", dense_args, dict(max_pages=1 << 28), INV), ("msa_dense_attn_decode_q8", dense_args, dict(seq_len=None), INV),
    ("msa_dense_attn_decode_q8", dense_args, dict(Q=FAKE + 4), INV), ("msa_dense_attn_decode_q8", dense_args, dict(window=-1), INV),
    ("msa_dense_attn_decode_q8", dense_args, dict(sinks=4), INV), ("msa_dense_attn_decode_q8", dense_args, dict(window=3, sinks=-1), INV),
    ("msa_window_attn_decode", window_args, dict(window=0), INV), ("msa_window_attn_decode", window_args, dict(sinks=-1), INV),
    ("msa_window_attn_decode", window_args, dict(B=1025), INV), ("msa_window_attn_decode", window_args, dict(Hq=18), UNS),
    ("msa_window_attn_decode", window_args, dict(Bk=64), UNS), ("msa_window_attn_decode", window_args, dict(D=64), UNS),
    ("msa_window_attn_decode", window_args, dict(kv_stride=(32768, 16384, 4)), INV), ("msa_window_attn_decode", window_args, dict(num_pages=0), INV),
    ("msa_window_attn_decode", window_args, dict(V_pool=None), INV), ("msa_window_attn_decode", window_args, dict(K_pool=FAKE + 8), INV),
    ("msa_window_attn_decode", window_args, dict(seq_pt=None), INV), ("msa_window_attn_decode", window_args, dict(max_pages=1 << 28), INV),
    ("msa_window_attn_prefill", prefill_args, dict(mode=1), INV), ("msa_window_attn_prefill", prefill_args, dict(window=0), INV),
    ("msa_window_attn_prefill", prefill_args, dict(sinks=-2), INV), ("msa_window_attn_prefill", prefill_args, dict(S=-1), INV),
    ("msa_window_attn_prefill", prefill_args, dict(Hq=18), UNS), ("msa_window_attn_prefill", prefill_args, dict(D=64), UNS),
    ("msa_window_attn_prefill", prefill_args, dict(B=1 << 20, S=1 << 20), UNS), ("msa_window_attn_prefill", prefill_args, dict(O=None), INV),
    ("msa_window_attn_prefill", prefill_args, dict(K=FAKE + 8), INV), ("msa_window_attn_prefill", prefill_args, dict(Q_stride=(61440, 1536, 4)), INV),
    ("msa_window_attn_prefill", chunk_args, dict(Bk=64), UNS), ("msa_window_attn_prefill", chunk_args, dict(seq_pt=None), INV),
    ("msa_window_attn_prefill", chunk_args, dict(q_pos=None), INV), ("msa_window_attn_prefill", chunk_args, dict(num_pages=0), INV),
    ("msa_window_attn_prefill", chunk_args, dict(max_pages=0), INV), ("msa_window_attn_prefill", chunk_args, dict(max_pages=(1 << 23) + 1), INV),
    ("msa_fork_requests", fork_args, dict(B=4097), UNS), ("msa_fork_requests", fork_args, dict(F=4097), UNS),
    ("msa_fork_requests", fork_args, dict(F=-1), UNS), ("msa_fork_requests", fork_args, dict(Bk=64), UNS),
    ("msa_fork_requests", fork_args, dict(num_pages=0), INV), ("msa_fork_requests", fork_args, dict(num_pages=(1 << 24) + 1), INV),
    ("msa_fork_requests", fork_args, dict(max_pages=0), INV), ("msa_fork_requests", fork_args, dict(free_cap=-1), INV),
    ("msa_fork_requests", fork_args, dict(F=4096, max_pages=1 << 20), UNS),
    ("msa_fork_requests", fork_args, dict(F=4096, max_pages=1 << 18), UNS),
    ("msa_compact_pages", compact_args, dict(B=4096, max_pages=1 << 18), UNS),
    ("msa_release_shared_pages", release_args, dict(B=4096, max_pages=1 << 18), UNS),
    *[("msa_fork_requests", fork_args, {n: None}, INV) for n in (
        "src", "dst", "seq_len", "seq_pt", "free_pages", "free_count", "page_shares", "seq_len_out", "seq_pt_out", "free_count_out",
        "page_shares_out", "copy_src", "copy_dst")],
    ("msa_release_shared_pages", release_args, dict(B=-1), UNS), ("msa_release_shared_pages", release_args, dict(B=4096, max_pages=1 << 20), UNS),
    ("msa_release_shared_pages", release_args, dict(num_pages=-3), INV),
    *[("msa_release_shared_pages", release_args, {n: None}, INV) for n in (
        "seq_len", "done", "seq_pt", "free_pages", "free_count", "page_shares", "seq_len_out", "free_count_out", "page_shares_out")],
    ("msa_compact_pages", compact_args, dict(free_cap=31), INV), ("msa_compact_pages", compact_args, dict(B=4097), UNS),
    ("msa_compact_pages", compact_args, dict(num_pages=0), INV),
    *[("msa_compact_pages", compact_args, {n: None}, INV) for n in (
        "seq_len", "seq_pt", "page_shares", "seq_pt_out", "page_shares_out", "free_pages", "free_count", "move_src", "move_dst")],
    ("msa_copy_pages", copy_args, dict(n=-1), INV), ("msa_copy_pages", copy_args, dict(num_pages=0), INV),
    ("msa_copy_pages", copy_args, dict(pools=17), UNS), ("msa_copy_pages", copy_args, dict(pools=-1), UNS),
    ("msa_copy_pages", copy_args, dict(pools=3), INV), ("msa_copy_pages", copy_args, dict(page_bytes=(513, 17)), INV),
    ("msa_copy_pages", copy_args, dict(page_bytes=(0, 17)), INV), ("msa_copy_pages", copy_args, dict(page_stride=(-512, 300)), INV),
    ("msa_copy_pages", copy_args, dict(src=None), INV), ("msa_copy_pages", copy_args, dict(dst=None), INV),
]


def call(abi, fn, a, ws_bytes=1 << 40, ws=FAKE):
    lib = abi.load()
    return getattr(lib, fn)(*((C.byref(a), ws, ws_bytes, None) if "attn_decode" in fn else (C.byref(a), None)))


@pytest.mark.parametrize("fn,build,kw,status", REFUSED, ids=[f"{f}-{next(iter(k))}{i}" for i, (f, _, k, _) in enumerate(REFUSED)])
def test_refused(abi, fn, build, kw, status):
    assert call(abi, fn, build(abi, **kw)) == status
    assert abi.load().msa_last_error_string()


@pytest.mark.parametrize("fn,build", [("msa_cache_append_q8", append_args), ("msa_cache_expand_q8", expand_args),
                                      ("msa_sparse_attn_decode_q8", sparse_args), ("msa_dense_attn_decode_q8", dense_args)])
def test_cache_refused(abi, fn, build):
    for kw in (dict(code_stride=(32768, 8)), dict(code_stride=(0, 16384)), dict(scale_stride=(0, 1)), dict(scale_stride=(2, -1)),
               dict(num_pages=0), dict(num_pages=1 << 31), dict(K_codes=None), dict(K_scales=None), dict(V_codes=FAKE + 8)):
        assert call(abi, fn, build(abi, cache=q8(abi, **kw))) == INV, kw


def test_workspace_refused(abi):
    lib = abi.load()
    need = lib.msa_attn_decode_q8_workspace_size(2, 2)
    assert need > 0 and lib.msa_window_attn_decode_workspace_size(2, 2) == need
    assert lib.msa_attn_decode_q8_workspace_size(-1, 2) == 0 and lib.msa_window_attn_decode_workspace_size(2, 0) == 0
    for fn, build in (("msa_sparse_attn_decode_q8", sparse_args), ("msa_dense_attn_decode_q8", dense_args), ("msa_window_attn_decode", window_args)):
        assert call(abi, fn, build(abi), need - 1) == WS
        assert call(abi, fn, build(abi), need, ws=None) == WS
        assert call(abi, fn, build(abi), need, ws=FAKE + 8) == INV


@pytest.mark.parametrize("fn", ["msa_cache_append_q8", "msa_cache_expand_q8", "msa_window_attn_prefill", "msa_fork_requests",
                                "msa_release_shared_pages", "msa_compact_pages", "msa_copy_pages"])
def test_null_args(abi, fn):
    assert getattr(abi.load(), fn)(None, None) == INV


def test_empty_calls_enqueue_nothing(abi):
    """And the pointer of an empty tensor is NULL."""
    for fn, a, names in (("msa_cache_append_q8", append_args(abi, N=0), ("K", "V", "slots")),
                         ("msa_cache_expand_q8", expand_args(abi, n=0), ("pages", "K_out", "V_out")),
                         ("msa_sparse_attn_decode_q8", sparse_args(abi, B=0), ("Q", "pt", "n", "last_len", "O", "LSE")),
                         ("msa_dense_attn_decode_q8", dense_args(abi, B=0), ("Q", "seq_pt", "seq_len", "O", "LSE")),
                         ("msa_window_attn_decode", window_args(abi, B=0), ("Q", "seq_pt", "seq_len", "O", "LSE")),
                         ("msa_window_attn_prefill", prefill_args(abi, B=0), ("Q", "K", "V", "O", "LSE")),
                         ("msa_window_attn_prefill", chunk_args(abi, S=0), ("Q", "O", "LSE")),
                         ("msa_copy_pages", copy_args(abi, n=0), ("src", "dst")), ("msa_copy_pages", copy_args(abi, pools=0), ())):
        assert call(abi, fn, a) == 0, fn
        for name in names:
            setattr(a, name, None)
        assert call(abi, fn, a) == 0, fn


# ---------------------------------------------------------------------------
# the Python wrappers
# ---------------------------------------------------------------------------

def wrapper_refusals(device):
    """Calls that the wrappers have to refuse, on tensors of this device."""
    import block_sparse_attention_02_gb300 as msa
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
    i32, i64, u8 = torch.int32, torch.int64, torch.uint8
    c = msa.q8_cache(3, 2, device)
    K, slots = z(4, 2, 128), z(4, dt=i64)
    L, pt, free, one = z(4, dt=i32), z(4, 2, dt=i32), z(9, dt=i32), z(1, dt=i32)
    Q, O, LSE, ws = z(2, 4, 128), z(2, 4, 128), z(2, 4, dt=torch.float32), z(64, dt=u8)
    pool, Qp, Kp = z(3, 2, 128, 128), z(2, 5, 4, 128), z(2, 5, 2, 128)
    Lp = z(2, 5, 4, dt=torch.float32)
    F = z(3, dt=i32)
    dense = lambda **k: msa.msa_dense_attn_decode_q8(**{**dict(Q=Q, cache=c, seq_pt=pt[:2], seq_len=L[:2], O=O, LSE=LSE, ws=ws), **k})  # noqa: E731
    window = lambda **k: msa.msa_window_attn_decode(**{**dict(  # noqa: E731
        Q=Q, K_pool=pool, V_pool=pool, seq_pt=pt[:2], seq_len=L[:2], O=O, LSE=LSE, ws=ws, window=5), **k})
    prefill = lambda **k: msa.msa_window_attn_prefill(**{**dict(Q=Qp, K=Kp, V=Kp, O=Qp, LSE=Lp, window=5), **k})  # noqa: E731
    fork = lambda **k: msa.msa_fork_requests(**{**dict(  # noqa: E731
        src=F, dst=F, seq_len=L, seq_pt=pt, free_pages=free, free_count=one, page_shares=free, seq_len_out=L, seq_pt_out=pt,
        free_count_out=one, page_shares_out=free, copy_src=F, copy_dst=F), **k})
    release = lambda **k: msa.msa_release_shared_pages(**{**dict(  # noqa: E731
        seq_len=L, done=L, seq_pt=pt, free_pages=free, free_count=one, page_shares=free, seq_len_out=L, free_count_out=one,
        page_shares_out=free), **k})
    compact = lambda **k: msa.msa_compact_pages(**{**dict(  # noqa: E731
        seq_len=L, seq_pt=pt, page_shares=free, seq_pt_out=pt, page_shares_out=free, free_pages=free, free_count=one, move_src=free,
        move_dst=free), **k})
    bad = [
        lambda: msa.msa_cache_append_q8(K, K, L, c), lambda: msa.msa_cache_append_q8(z(4, 3, 128), z(4, 3, 128), slots, c),
        lambda: msa.msa_cache_append_q8(K, K[:3], slots, c), lambda: msa.msa_cache_append_q8(K, K, slots, c._replace(V_codes=c.V_codes[:2])),
        lambda: msa.msa_cache_append_q8(K, K, slots, c._replace(K_scales=c.K_scales[:, :1])),
        lambda: msa.msa_cache_append_q8(K, K, slots, c._replace(K_scales=c.K_scales.float())),
        lambda: msa.msa_cache_append_q8(K, K, slots, c._replace(K_codes=z(3, 128, 2, 128, dt=u8).transpose(1, 2))),
        lambda: msa.msa_cache_append_q8(K, K, slots, c._replace(V_scales=z(2, 3, dt=u8).T)),
        lambda: msa.msa_cache_append_q8(K, K, slots, c[:3]), lambda: msa.msa_cache_append_q8(K, K, slots, msa.q4_cache(3, 2, device)),
        lambda: msa.msa_cache_append_q8(K.float(), K.float(), slots, c),
        lambda: msa.msa_cache_expand_q8(c, one, z(1, 2, 128, 128), z(2, 2, 128, 128)),
        lambda: msa.msa_sparse_attn_decode_q8(Q, c, pt[:3], L, L, O, LSE, ws), lambda: msa.msa_sparse_attn_decode_q8(Q, c, pt, L, L, O[:1], LSE, ws),
        lambda: dense(seq_len=L), lambda: dense(ws=z(128, dt=u8)[::2]), lambda: dense(LSE=LSE[:1]), lambda: dense(window=1.5), lambda: dense(window=1 << 40),
        lambda: dense(sinks="x"), lambda: dense(cache=msa.q4_cache(3, 2, device)),
        lambda: window(V_pool=z(3, 2, 64, 128)), lambda: window(K_pool=pool.float()), lambda: window(K_pool=z(3, 2, 128, 64)),
        lambda: window(V_pool=z(3, 2, 128, 256)[..., ::2]), lambda: window(V_pool=z(3, 2, 128, 256)[..., :128]), lambda: window(seq_pt=pt),
        lambda: window(window="x"),
        lambda: prefill(K=Kp[:1]), lambda: prefill(V=z(2, 5, 1, 128)), lambda: prefill(O=Qp[:, :4]), lambda: prefill(LSE=LSE), lambda: prefill(seq_pt=pt[:2]),
        lambda: prefill(q_pos=L[:2]), lambda: prefill(seq_pt=pt, q_pos=L[:2], K=pool, V=pool), lambda: prefill(seq_pt=pt[:2], q_pos=L, K=pool, V=pool),
        lambda: prefill(seq_pt=pt[:2], q_pos=L[:2]), lambda: prefill(Q=Qp.float()), lambda: prefill(O=z(2, 4, 5, 128).transpose(1, 2)),
        lambda: prefill(window=1 << 31),
        lambda: fork(dst=L), lambda: fork(src=F.long()), lambda: fork(seq_pt_out=z(4, 3, dt=i32)), lambda: fork(seq_pt=z(2, 4, dt=i32).T),
        lambda: fork(page_shares_out=one), lambda: fork(copy_dst=L), lambda: fork(free_count=F), lambda: fork(seq_len_out=F),
        lambda: fork(dev_err=z(0, dt=i32)), lambda: fork(stream="s"),
        lambda: release(done=F), lambda: release(done=L.bool()), lambda: release(page_shares_out=L), lambda: release(seq_len_out=F),
        lambda: compact(seq_pt_out=pt[:3]), lambda: compact(move_src=L), lambda: compact(page_shares=free.long()), lambda: compact(free_count=F),
        lambda: msa.msa_copy_pages([pool, z(4, 2)], F, F), lambda: msa.msa_copy_pages([pool.transpose(1, 2)], F, F),
        lambda: msa.msa_copy_pages(pool, F, F), lambda: msa.msa_copy_pages([pool], F, L), lambda: msa.msa_copy_pages([pool] * 17, F, F),
        lambda: msa.msa_copy_pages([3], F, F), lambda: msa.msa_copy_pages([z(0, 2)], F, F), lambda: msa.msa_copy_pages([pool], F.long(), F.long()),
        lambda: msa.msa_copy_pages([z(2, 6)[:, ::2]], F, F),
    ]
    on_host_only = [lambda: msa.msa_cache_append_q8(K, K, slots, c), lambda: msa.msa_cache_expand_q8(c, one, z(1, 2, 128, 128), z(1, 2, 128, 128)),
                    lambda: msa.msa_sparse_attn_decode_q8(Q, c, pt, L, L, O, LSE, ws), dense, window, prefill, fork, release, compact,
                    lambda: msa.msa_copy_pages([pool], F, F)]
    return bad + (on_host_only if device == "cpu" else [])


def test_wrappers_refuse(abi):
    for i, refused in enumerate(wrapper_refusals("cpu")):
        with pytest.raises(ValueError):
            refused()
            raise AssertionError(f"call {i} was accepted")


@pytest.mark.gpu
def test_wrappers_refuse_on_the_gpu(abi):
    for i, refused in enumerate(wrapper_refusals("cuda")):
        with pytest.raises(ValueError):
            refused()
            raise AssertionError(f"call {i} was accepted")
