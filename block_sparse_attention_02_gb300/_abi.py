"""ctypes mirror of include/msa.h and the loader of libmsa.so.

Nothing here computes: it declares the C structs and function signatures and
loads the in-tree library built by ``build.py``.  There is no fallback; if the
library is missing the import of the binding raises.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmsa.so")

MSA_OK = 0
MSA_ERR_INVALID_ARG = 1
MSA_ERR_UNSUPPORTED = 2
MSA_ERR_CUDA = 3
MSA_ERR_DEVICE_CHECK = 4
MSA_ERR_WORKSPACE = 5

MSA_DEVERR_TIMEOUT = 0x1
MSA_DEVERR_BAD_PAGE = 0x2
MSA_DEVERR_BAD_SEL = 0x4
MSA_DEVERR_BAD_LEN = 0x8
MSA_DEVERR_NO_PAGES = 0x10

MSA_MODE_PREFILL = 0
MSA_MODE_DECODE = 1
MSA_MODE_CHUNK = 2

_p = C.c_void_p
_i64x2 = C.c_int64 * 2
_i64x3 = C.c_int64 * 3
_i64x4 = C.c_int64 * 4


class IndexArgs(C.Structure):
    _fields_ = [
        ("mode", C.c_int), ("B", C.c_int), ("S", C.c_int), ("Hkv", C.c_int), ("HI", C.c_int),
        ("dI", C.c_int), ("Bk", C.c_int),
        ("q_idx", _p), ("q_idx_stride", _i64x4),
        ("w", _p), ("w_stride", _i64x3),
        ("k_idx", _p), ("k_idx_stride", _i64x3),
        ("num_pages", C.c_int64), ("seq_pt", _p), ("max_pages", C.c_int64), ("seq_len", _p),
        ("C", _p), ("C_stride", _i64x3), ("nb_stride", C.c_int),
        ("dev_err", _p),
        ("k", C.c_int), ("sel", _p), ("count", _p), ("pt", _p), ("n", _p), ("last_len", _p),
        ("row_scratch", _p), ("scratch_zeroed", C.c_int),
        ("q_pos", _p),
    ]


class TopkArgs(C.Structure):
    _fields_ = [
        ("mode", C.c_int), ("B", C.c_int), ("S", C.c_int), ("Hkv", C.c_int), ("Bk", C.c_int), ("k", C.c_int),
        ("C", _p), ("C_stride", _i64x3), ("nb_stride", C.c_int),
        ("seq_len", _p), ("sel", _p), ("count", _p), ("dev_err", _p),
        ("q_pos", _p),
    ]


class PrefillArgs(C.Structure):
    _fields_ = [
        ("B", C.c_int), ("S", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("Bk", C.c_int),
        ("k", C.c_int), ("softmax_scale", C.c_float),
        ("Q", _p), ("Q_stride", _i64x3), ("K", _p), ("K_stride", _i64x3), ("V", _p), ("V_stride", _i64x3),
        ("sel", _p), ("count", _p), ("O", _p), ("LSE", _p), ("dev_err", _p),
        ("mode", C.c_int), ("seq_pt", _p), ("max_pages", C.c_int64), ("num_pages", C.c_int64), ("q_pos", _p),
    ]


class DecodeArgs(C.Structure):
    _fields_ = [
        ("B", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("Bk", C.c_int), ("k", C.c_int),
        ("softmax_scale", C.c_float),
        ("Q", _p), ("Q_stride", _i64x2), ("K_pool", _p), ("V_pool", _p), ("kv_stride", _i64x3),
        ("num_pages", C.c_int64), ("pt", _p), ("n", _p), ("last_len", _p),
        ("O", _p), ("LSE", _p), ("dev_err", _p), ("scratch_zeroed", C.c_int),
    ]


class AppendArgs(C.Structure):
    _fields_ = [
        ("B", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("dI", C.c_int), ("Bk", C.c_int),
        ("K_new", _p), ("K_new_stride", _i64x2), ("V_new", _p), ("V_new_stride", _i64x2),
        ("kidx_new", _p), ("kidx_new_stride", _i64x2),
        ("K_pool", _p), ("V_pool", _p), ("kv_stride", _i64x3), ("kidx_pool", _p), ("kidx_stride", _i64x3),
        ("num_pages", C.c_int64), ("seq_pt", _p), ("max_pages", C.c_int64), ("seq_len", _p), ("dev_err", _p),
        ("T", C.c_int), ("new_t_stride", _i64x3),
    ]


class DenseDecodeArgs(C.Structure):
    _fields_ = [
        ("B", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("Bk", C.c_int),
        ("softmax_scale", C.c_float),
        ("Q", _p), ("Q_stride", _i64x2), ("K_pool", _p), ("V_pool", _p), ("kv_stride", _i64x3),
        ("num_pages", C.c_int64), ("seq_pt", _p), ("max_pages", C.c_int64), ("seq_len", _p),
        ("O", _p), ("LSE", _p), ("dev_err", _p), ("scratch_zeroed", C.c_int),
    ]


class DensePrefillArgs(C.Structure):
    _fields_ = [
        ("B", C.c_int), ("S", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int),
        ("softmax_scale", C.c_float),
        ("Q", _p), ("Q_stride", _i64x3), ("K", _p), ("K_stride", _i64x3), ("V", _p), ("V_stride", _i64x3),
        ("O", _p), ("LSE", _p), ("dev_err", _p),
    ]


class PlanArgs(C.Structure):
    _fields_ = [
        ("B", C.c_int), ("Bk", C.c_int), ("N", C.c_int64),
        ("seq_len", _p), ("new_len", _p), ("seq_pt", _p), ("max_pages", C.c_int64),
        ("free_pages", _p), ("free_cap", C.c_int64), ("free_count", _p), ("num_pages", C.c_int64),
        ("seq_len_out", _p), ("free_count_out", _p), ("cu", _p),
        ("tok_slot", _p), ("tok_pos", _p), ("tok_seq", _p), ("dev_err", _p),
    ]


class ReleaseArgs(C.Structure):
    _fields_ = [
        ("B", C.c_int), ("Bk", C.c_int), ("seq_len", _p), ("done", _p), ("seq_pt", _p), ("max_pages", C.c_int64),
        ("free_pages", _p), ("free_cap", C.c_int64), ("free_count", _p),
        ("seq_len_out", _p), ("free_count_out", _p), ("dev_err", _p), ("num_pages", C.c_int64),
    ]


class NormRopeArgs(C.Structure):
    _fields_ = [
        ("N", C.c_int64), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("Bk", C.c_int), ("rot", C.c_int),
        ("interleaved", C.c_int), ("weight_fp32", C.c_int), ("eps", C.c_float),
        ("Q", _p), ("Q_stride", _i64x2), ("K", _p), ("K_stride", _i64x2), ("V", _p), ("V_stride", _i64x2),
        ("pos", _p), ("inv_freq", _p), ("q_weight", _p), ("k_weight", _p),
        ("Q_out", _p), ("Q_out_stride", _i64x2), ("K_out", _p), ("K_out_stride", _i64x3),
        ("V_out", _p), ("V_out_stride", _i64x3), ("slots", _p), ("num_pages", C.c_int64), ("dev_err", _p),
    ]


class Q4CacheArgs(C.Structure):
    _fields_ = [
        ("K_codes", _p), ("K_scales", _p), ("V_codes", _p), ("V_scales", _p),
        ("code_stride", _i64x2), ("scale_stride", _i64x2), ("num_pages", C.c_int64),
        ("k_scale", C.c_float), ("v_scale", C.c_float),
    ]


class AppendQ4Args(C.Structure):
    _fields_ = [
        ("N", C.c_int64), ("Hkv", C.c_int), ("D", C.c_int), ("Bk", C.c_int),
        ("K", _p), ("K_stride", _i64x2), ("V", _p), ("V_stride", _i64x2), ("slots", _p),
        ("cache", Q4CacheArgs), ("dev_err", _p),
    ]


class ExpandQ4Args(C.Structure):
    _fields_ = [
        ("n", C.c_int64), ("Hkv", C.c_int), ("D", C.c_int), ("Bk", C.c_int), ("pages", _p),
        ("cache", Q4CacheArgs), ("K_out", _p), ("V_out", _p), ("dev_err", _p),
    ]


class DecodeQ4Args(C.Structure):
    _fields_ = [
        ("B", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("Bk", C.c_int), ("k", C.c_int),
        ("softmax_scale", C.c_float), ("Q", _p), ("Q_stride", _i64x2), ("cache", Q4CacheArgs),
        ("pt", _p), ("n", _p), ("last_len", _p), ("O", _p), ("LSE", _p), ("dev_err", _p), ("scratch_zeroed", C.c_int),
    ]


class DenseDecodeQ4Args(C.Structure):
    _fields_ = [
        ("B", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("Bk", C.c_int),
        ("softmax_scale", C.c_float), ("Q", _p), ("Q_stride", _i64x2), ("cache", Q4CacheArgs),
        ("seq_pt", _p), ("max_pages", C.c_int64), ("seq_len", _p),
        ("O", _p), ("LSE", _p), ("dev_err", _p), ("scratch_zeroed", C.c_int),
    ]


# exported function name -> (restype, argtypes)
SIGNATURES = {
    "msa_version": (C.c_int, []),
    "msa_last_error_string": (C.c_char_p, []),
    "msa_status_string": (C.c_char_p, [C.c_int]),
    "msa_index_score": (C.c_int, [C.POINTER(IndexArgs), _p]),
    "msa_topk_blocks": (C.c_int, [C.POINTER(TopkArgs), _p]),
    "msa_build_page_table": (C.c_int, [_p, _p, _p, C.c_int64, _p, C.c_int, C.c_int, C.c_int, C.c_int,
                                       _p, _p, _p, _p, _p]),
    "msa_sparse_attn_prefill_workspace_size": (C.c_size_t, [C.POINTER(PrefillArgs), C.c_int64]),
    "msa_sparse_attn_prefill": (C.c_int, [C.POINTER(PrefillArgs), _p, C.c_size_t, _p]),
    "msa_sparse_attn_decode_workspace_size": (C.c_size_t, [C.POINTER(DecodeArgs)]),
    "msa_sparse_attn_decode": (C.c_int, [C.POINTER(DecodeArgs), _p, C.c_size_t, _p]),
    "msa_sparse_attn_decode_noalloc": (C.c_int, [C.POINTER(DecodeArgs), _p]),
    "msa_lse_merge": (C.c_int, [_p, _p, C.c_int64, C.c_int, C.c_int, _p, _p, _p, _p]),
    "msa_cache_append": (C.c_int, [C.POINTER(AppendArgs), _p]),
    "msa_dense_attn_decode_workspace_size": (C.c_size_t, [C.POINTER(DenseDecodeArgs)]),
    "msa_dense_attn_decode": (C.c_int, [C.POINTER(DenseDecodeArgs), _p, C.c_size_t, _p]),
    "msa_dense_attn_prefill": (C.c_int, [C.POINTER(DensePrefillArgs), _p]),
    "msa_plan_step": (C.c_int, [C.POINTER(PlanArgs), _p]),
    "msa_release_pages": (C.c_int, [C.POINTER(ReleaseArgs), _p]),
    "msa_qk_norm_rope": (C.c_int, [C.POINTER(NormRopeArgs), _p]),
    "msa_cache_append_q4": (C.c_int, [C.POINTER(AppendQ4Args), _p]),
    "msa_cache_expand_q4": (C.c_int, [C.POINTER(ExpandQ4Args), _p]),
    "msa_attn_decode_q4_workspace_size": (C.c_size_t, [C.c_int, C.c_int]),
    "msa_sparse_attn_decode_q4": (C.c_int, [C.POINTER(DecodeQ4Args), _p, C.c_size_t, _p]),
    "msa_dense_attn_decode_q4": (C.c_int, [C.POINTER(DenseDecodeQ4Args), _p, C.c_size_t, _p]),
}

_lock = threading.Lock()
_lib = None
_binding = None


def load(path: str = LIB_PATH):
    """Load libmsa.so (built in-tree); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
            lib = C.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(lib, name)
                f.restype = res
                f.argtypes = args
            _lib = lib
    return _lib


def binding():
    """The module that marshals torch tensors for the serving-step calls (built in-tree beside libmsa.so)."""
    global _binding
    if _binding is None:
        load()
        try:
            from . import _msa_binding
        except ImportError as e:
            raise RuntimeError("_msa_binding is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`") from e
        import torch
        if _msa_binding.built_for != str(torch.__version__):
            raise RuntimeError(f"_msa_binding was built for torch {_msa_binding.built_for}, this is {torch.__version__}: build it "
                               "again with `python -c 'import __graft_entry__ as g; g.build()'`")
        _binding = _msa_binding
    return _binding


class MSAError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        self.status = status
        name = load().msa_status_string(status).decode()
        super().__init__(f"{func}: {name}: {detail}")


def check(status: int, func: str) -> None:
    if status != MSA_OK:
        raise MSAError(status, func, load().msa_last_error_string().decode())
