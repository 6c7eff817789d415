"""Refusals of the serving-step entry points without a GPU: struct layouts, argument checks of the C calls (nothing is
enqueued) and of the Python wrappers."""
import ctypes as C
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def abi():
    from block_sparse_attention_02_gb300 import build as b
    b.build()
    from block_sparse_attention_02_gb300 import _abi
    _abi.load()
    return _abi


def test_struct_layout_matches_header(abi, tmp_path):
    structs = {"msa_plan_args": abi.PlanArgs, "msa_release_args": abi.ReleaseArgs, "msa_norm_rope_args": abi.NormRopeArgs,
               "msa_q4_cache": abi.Q4CacheArgs, "msa_append_q4_args": abi.AppendQ4Args, "msa_expand_q4_args": abi.ExpandQ4Args,
               "msa_decode_q4_args": abi.DecodeQ4Args, "msa_dense_decode_q4_args": abi.DenseDecodeQ4Args}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "msa.h"', "int main(void) {"]
    for c, py in structs.items():
        lines.append(f'printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
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
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def plan_args(abi, **kw):
    return make(abi.PlanArgs, **{**dict(B=4, Bk=128, N=16, max_pages=8, free_cap=32, num_pages=32), **kw})


def release_args(abi, **kw):
    return make(abi.ReleaseArgs, **{**dict(B=4, Bk=128, max_pages=8, free_cap=32), **kw})


def rope_args(abi, **kw):
    return make(abi.NormRopeArgs, **{**dict(
        N=4, Hq=4, Hkv=2, D=128, Bk=128, rot=128, eps=1e-6, Q_stride=(1024, 128), K_stride=(1024, 128), V_stride=(1024, 128),
        Q_out_stride=(512, 128), K_out_stride=(32768, 16384, 128), V_out_stride=(32768, 16384, 128), num_pages=9), **kw})


def q4(abi, **kw):
    return make(abi.Q4CacheArgs, **{**dict(code_stride=(16384, 8192), scale_stride=(2048, 1024), num_pages=9, k_scale=1.0,
                                           v_scale=0.5), **kw})


def append_args(abi, cache=None, **kw):
    return make(abi.AppendQ4Args, **{**dict(N=4, Hkv=2, D=128, Bk=128, K_stride=(256, 128), V_stride=(256, 128)), **kw,
                                     "cache": cache or q4(abi)})


def expand_args(abi, cache=None, **kw):
    return make(abi.ExpandQ4Args, **{**dict(n=4, Hkv=2, D=128, Bk=128), **kw, "cache": cache or q4(abi)})


def sparse_args(abi, cache=None, **kw):
    return make(abi.DecodeQ4Args, **{**dict(B=2, Hq=12, Hkv=2, D=128, Bk=128, k=16, Q_stride=(1536, 128)), **kw,
                                     "cache": cache or q4(abi)})


def dense_args(abi, cache=None, **kw):
    return make(abi.DenseDecodeQ4Args, **{**dict(B=2, Hq=12, Hkv=2, D=128, Bk=128, Q_stride=(1536, 128), max_pages=8), **kw,
                                          "cache": cache or q4(abi)})


INV, UNS, WS = 1, 2, 5
REFUSED = [
    ("msa_plan_step", plan_args, dict(B=-1), UNS), ("msa_plan_step", plan_args, dict(B=4097), UNS),
    ("msa_plan_step", plan_args, dict(Bk=64), UNS), ("msa_plan_step", plan_args, dict(max_pages=0), INV),
    ("msa_plan_step", plan_args, dict(max_pages=1 << 24), INV), ("msa_plan_step", plan_args, dict(N=-1), INV),
    ("msa_plan_step", plan_args, dict(N=(1 << 31) - 1), INV), ("msa_plan_step", plan_args, dict(free_cap=-1), INV),
    ("msa_plan_step", plan_args, dict(num_pages=0), INV), ("msa_plan_step", plan_args, dict(seq_len=None), INV),
    ("msa_plan_step", plan_args, dict(new_len=None), INV), ("msa_plan_step", plan_args, dict(seq_pt=None), INV),
    ("msa_plan_step", plan_args, dict(free_pages=None), INV), ("msa_plan_step", plan_args, dict(free_count=None), INV),
    ("msa_plan_step", plan_args, dict(cu=None), INV), ("msa_plan_step", plan_args, dict(tok_slot=None), INV),
    ("msa_plan_step", plan_args, dict(tok_pos=None), INV),
    ("msa_release_pages", release_args, dict(B=4097), UNS), ("msa_release_pages", release_args, dict(Bk=256), UNS),
    ("msa_release_pages", release_args, dict(done=None), INV), ("msa_release_pages", release_args, dict(free_count_out=None), INV),
    ("msa_qk_norm_rope", rope_args, dict(D=96), UNS), ("msa_qk_norm_rope", rope_args, dict(rot=24), UNS),
    ("msa_qk_norm_rope", rope_args, dict(rot=144), UNS), ("msa_qk_norm_rope", rope_args, dict(N=-1), INV),
    ("msa_qk_norm_rope", rope_args, dict(eps=-1.0), INV), ("msa_qk_norm_rope", rope_args, dict(eps=float("nan")), INV),
    ("msa_qk_norm_rope", rope_args, dict(pos=None), INV), ("msa_qk_norm_rope", rope_args, dict(inv_freq=None), INV),
    ("msa_qk_norm_rope", rope_args, dict(Q_out=None), INV), ("msa_qk_norm_rope", rope_args, dict(K_out=None), INV),
    ("msa_qk_norm_rope", rope_args, dict(V_out=None), INV), ("msa_qk_norm_rope", rope_args, dict(slots=None), INV),
    ("msa_qk_norm_rope", rope_args, dict(Q=FAKE + 8), INV), ("msa_qk_norm_rope", rope_args, dict(Q_stride=(1020, 128)), INV),
    ("msa_qk_norm_rope", rope_args, dict(K_stride=(0, 128)), INV), ("msa_qk_norm_rope", rope_args, dict(num_pages=0), INV),
    ("msa_qk_norm_rope", rope_args, dict(V_out_stride=(32768, 16384, 4)), INV), ("msa_qk_norm_rope", rope_args, dict(Bk=64), UNS),
    ("msa_cache_append_q4", append_args, dict(D=64), UNS), ("msa_cache_append_q4", append_args, dict(Bk=64), UNS),
    ("msa_cache_append_q4", append_args, dict(N=-1), INV), ("msa_cache_append_q4", append_args, dict(Hkv=0), INV),
    ("msa_cache_append_q4", append_args, dict(slots=None), INV), ("msa_cache_append_q4", append_args, dict(V_stride=(256, 4)), INV),
    ("msa_cache_append_q4", append_args, dict(K=FAKE + 2), INV),
    ("msa_cache_expand_q4", expand_args, dict(n=-1), INV), ("msa_cache_expand_q4", expand_args, dict(pages=None), INV),
    ("msa_cache_expand_q4", expand_args, dict(V_out=FAKE + 8), INV),
    ("msa_sparse_attn_decode_q4", sparse_args, dict(B=4097), INV), ("msa_sparse_attn_decode_q4", sparse_args, dict(k=65), UNS),
    ("msa_sparse_attn_decode_q4", sparse_args, dict(B=4096, Hq=1 << 15, Hkv=1 << 13), UNS),
    ("msa_sparse_attn_decode_q4", sparse_args, dict(k=0), UNS), ("msa_sparse_attn_decode_q4", sparse_args, dict(Hq=18), UNS),
    ("msa_sparse_attn_decode_q4", sparse_args, dict(Hq=13), UNS), ("msa_sparse_attn_decode_q4", sparse_args, dict(D=64), UNS),
    ("msa_sparse_attn_decode_q4", sparse_args, dict(pt=None), INV), ("msa_sparse_attn_decode_q4", sparse_args, dict(O=None), INV),
    ("msa_sparse_attn_decode_q4", sparse_args, dict(Q_stride=(1536, 100)), INV),
    ("msa_dense_attn_decode_q4", dense_args, dict(B=1025), INV), ("msa_dense_attn_decode_q4", dense_args, dict(max_pages=0), INV),
    ("msa_dense_attn_decode_q4", dense_args, dict(max_pages=1 << 28), INV), ("msa_dense_attn_decode_q4", dense_args, dict(seq_len=None), INV),
    ("msa_dense_attn_decode_q4", dense_args, dict(Q=FAKE + 4), INV),
]


def test_store_rounding_of_every_value():
    """The store's fp32 steps against the definition, for every bf16 magnitude up to past the range under every scale:
    x r + 1536 in one rounding, less 1536, then the nearest code; and amax / 6 as a product."""
    import numpy as np
    import serving_ref as ref
    x = (np.arange(1, 0x7F80, dtype=np.uint32) << 16).view(np.float32)
    for step in ref.E4M3[1:].astype(np.float32):
        v = x[x <= step * np.float32(7.5)].astype(np.float64)
        q = (v * np.float64(np.float32(1) / step) + 1536.0).astype(np.float32) - np.float32(1536)
        assert np.array_equal(ref.nearest(ref.GRID, np.minimum(q.astype(np.float64), 6.0)),
                              ref.nearest(ref.GRID, np.minimum(v / np.float64(step), 6.0))), step
    a = x[x <= 2688]
    assert np.array_equal(ref.nearest(ref.E4M3, (a * np.float32(1 / 6)).astype(np.float64)),
                          ref.nearest(ref.E4M3, a.astype(np.float64) / 6))


def call(abi, fn, a, ws_bytes=1 << 40, ws=FAKE):
    lib = abi.load()
    return getattr(lib, fn)(*((C.byref(a), ws, ws_bytes, None) if "attn" in fn else (C.byref(a), None)))


@pytest.mark.parametrize("fn,build,kw,status", REFUSED, ids=[f"{f}-{next(iter(k))}{i}" for i, (f, _, k, _) in enumerate(REFUSED)])
def test_refused(abi, fn, build, kw, status):
    assert call(abi, fn, build(abi, **kw)) == status
    assert abi.load().msa_last_error_string()


@pytest.mark.parametrize("fn,build", [("msa_cache_append_q4", append_args), ("msa_cache_expand_q4", expand_args),
                                      ("msa_sparse_attn_decode_q4", sparse_args), ("msa_dense_attn_decode_q4", dense_args)])
def test_cache_refused(abi, fn, build):
    for kw in (dict(k_scale=0.0), dict(k_scale=3.0), dict(v_scale=-1.0), dict(v_scale=float("inf")), dict(k_scale=float("nan")),
               dict(k_scale=2.0 ** 65), dict(v_scale=2.0 ** -65), dict(code_stride=(16384, 8)), dict(scale_stride=(0, 1024)), dict(code_stride=(1 << 32, 8192)),
               dict(num_pages=0), dict(K_codes=None), dict(V_scales=FAKE + 8)):
        assert call(abi, fn, build(abi, cache=q4(abi, **kw))) == INV, kw


def test_workspace_refused(abi):
    need = abi.load().msa_attn_decode_q4_workspace_size(2, 2)
    assert need > 0 and abi.load().msa_attn_decode_q4_workspace_size(-1, 2) == 0
    for fn, build in (("msa_sparse_attn_decode_q4", sparse_args), ("msa_dense_attn_decode_q4", dense_args)):
        assert call(abi, fn, build(abi), need - 1) == WS
        assert call(abi, fn, build(abi), need, ws=None) == WS
        assert call(abi, fn, build(abi), need, ws=FAKE + 8) == INV


@pytest.mark.parametrize("fn", ["msa_plan_step", "msa_release_pages", "msa_qk_norm_rope", "msa_cache_append_q4", "msa_cache_expand_q4"])
def test_null_args(abi, fn):
    assert getattr(abi.load(), fn)(None, None) == INV


def test_empty_calls_enqueue_nothing(abi):
    for fn, a in (("msa_qk_norm_rope", rope_args(abi, N=0)), ("msa_cache_append_q4", append_args(abi, N=0)),
                  ("msa_cache_expand_q4", expand_args(abi, n=0)), ("msa_sparse_attn_decode_q4", sparse_args(abi, B=0)),
                  ("msa_dense_attn_decode_q4", dense_args(abi, B=0))):
        assert call(abi, fn, a) == 0, fn


def test_empty_calls_need_no_rows(abi):
    """The pointer of an empty tensor is NULL."""
    for fn, a, names in (("msa_qk_norm_rope", rope_args(abi, N=0), ("pos", "Q", "K", "Q_out")),
                         ("msa_cache_append_q4", append_args(abi, N=0), ("K", "V", "slots")),
                         ("msa_cache_expand_q4", expand_args(abi, n=0), ("pages", "K_out", "V_out")),
                         ("msa_sparse_attn_decode_q4", sparse_args(abi, B=0), ("Q", "pt", "n", "last_len", "O", "LSE")),
                         ("msa_dense_attn_decode_q4", dense_args(abi, B=0), ("Q", "seq_pt", "seq_len", "O", "LSE"))):
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
    i32, i64 = torch.int32, torch.int64
    c = msa.q4_cache(3, 2, device)
    Q, K, pos = z(4, 6, 128), z(4, 2, 128), z(4, dt=i32)
    L, pt, free, one = z(4, dt=i32), z(4, 2, dt=i32), z(9, dt=i32), z(1, dt=i32)
    rows, rows32 = z(5, dt=i64), z(5, dt=i32)
    O, LSE, ws, f = z(2, 4, 128), z(2, 4, dt=torch.float32), z(64, dt=torch.uint8), z(64, dt=torch.float32)
    plan = lambda **k: msa.msa_plan_step(**{**dict(  # noqa: E731
        seq_len=L, new_len=L, seq_pt=pt, free_pages=free, free_count=one, seq_len_out=L, free_count_out=one,
        cu=rows32, tok_slot=rows, tok_pos=rows32, num_pages=9), **k})
    rope = lambda **k: msa.msa_qk_norm_rope(**{**dict(Q=Q, K=K, pos=pos, inv_freq=f, Q_out=Q, K_out=K), **k})  # noqa: E731
    bad = [
        lambda: plan(new_len=z(3, dt=i32)), lambda: plan(cu=L), lambda: plan(tok_pos=L), lambda: plan(seq_len=z(4, dt=i64)),
        lambda: plan(seq_pt=z(2, 4, dt=i32).T), lambda: plan(free_count=z(2, dt=i32)), lambda: plan(tok_seq=z(6, dt=i32)),
        lambda: plan(dev_err=z(0, dt=i32)), lambda: plan(dev_err=z(1, dt=i64)),
        lambda: msa.msa_release_pages(L, L[:3], pt, free, one, L, one), lambda: msa.msa_release_pages(L, L.bool(), pt, free, one, L, one),
        lambda: rope(Q_out=z(4, 5, 128)), lambda: rope(K=None), lambda: rope(K_out=z(3, 2, 128, 128)), lambda: rope(pos=pos[:3]),
        lambda: rope(V=K), lambda: rope(slots=z(4, dt=i64)), lambda: rope(q_weight=z(64)), lambda: rope(q_weight=z(128, dt=torch.float16)),
        lambda: rope(q_weight=z(128), k_weight=z(128, dt=torch.float32)), lambda: rope(Q=z(4, 6, 256)[..., ::2], Q_out=Q),
        lambda: rope(inv_freq=f.double()), lambda: rope(Q=Q.float()), lambda: rope(K_out=z(3, 2, 64, 128), slots=z(4, dt=i64)),
        lambda: msa.msa_cache_append_q4(K, K, z(4, dt=i32), c),
        lambda: msa.msa_cache_append_q4(z(4, 3, 128), z(4, 3, 128), z(4, dt=i64), c), lambda: msa.msa_cache_append_q4(K, K[:3], z(4, dt=i64), c),
        lambda: msa.msa_cache_append_q4(K, K, z(4, dt=i64), c._replace(V_codes=c.V_codes[:2])),
        lambda: msa.msa_cache_append_q4(K, K, z(4, dt=i64), c._replace(K_codes=z(3, 128, 2, 64, dt=torch.uint8).transpose(1, 2))),
        lambda: msa.msa_cache_expand_q4(c, one, z(1, 2, 128, 128), z(2, 2, 128, 128)),
        lambda: msa.msa_sparse_attn_decode_q4(O, c, pt[:3], L, L, O, LSE, ws),
        lambda: msa.msa_sparse_attn_decode_q4(O, c, pt, L, L, O[:1], LSE, ws), lambda: msa.msa_sparse_attn_decode_q4(O, c, pt, L, L, O, LSE[:1], ws),
        lambda: msa.msa_dense_attn_decode_q4(O, c, pt, L, O, LSE, ws),
        lambda: msa.msa_dense_attn_decode_q4(O, c, pt[:2], L[:2], O, LSE, ws[::2]),
        lambda: rope(inv_freq=z(68, dt=torch.float32)[::2]), lambda: plan(stream="s"), lambda: plan(num_pages=2.5),
        lambda: msa.msa_cache_append_q4(K, K, z(4, dt=i64), c[:4]), lambda: msa.msa_cache_append_q4([], K, z(4, dt=i64), c),
        lambda: msa.msa_cache_append_q4(K, K, z(4, dt=i64), c._replace(k_scale="x")),
    ]
    on_host_only = [plan, lambda: msa.msa_release_pages(L, L, pt, free, one, L, one), rope,
                    lambda: msa.msa_cache_append_q4(K, K, z(4, dt=i64), c),
                    lambda: msa.msa_cache_expand_q4(c, one, z(1, 2, 128, 128), z(1, 2, 128, 128)),
                    lambda: msa.msa_sparse_attn_decode_q4(O, c, pt, L, L, O, LSE, ws),
                    lambda: msa.msa_dense_attn_decode_q4(O, c, pt[:2], L[:2], O, LSE, ws)]
    return bad + (on_host_only if device == "cpu" else [])


def test_wrappers_refuse(abi):
    for i, refused in enumerate(wrapper_refusals("cpu")):
        with pytest.raises(ValueError):
            refused()
            raise AssertionError(f"call {i} was accepted")
