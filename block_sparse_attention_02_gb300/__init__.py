"""MiniMax Sparse Attention (MSA) hot path on one GB300 -- Python binding.

Marshalling over ``libmsa.so`` (include/msa.h), in ctypes or C++.  Every function
takes torch CUDA tensors, passes their pointers and element strides to the C
entry point of the same name, and raises ``MSAError`` on a non-OK status.  All
computation runs in the library's sm_103a kernels; there is no fallback path.
PyTorch provides device memory and streams only.  The calls of the serving step around the
cache (page tables, norm with rotation, the 4-bit and 8-bit caches and their attention) go through a module in
C++ (``_msa_binding``): their kernels take a few microseconds, and so would Python on their arguments.

The pipelines at the bottom (``decode_step``, ``decode_step_q4``, ``decode_step_q8``, ``prefill_layer``
and ``chunk_layer``) call the entry points in hot-path order: index score -> top-k
-> (decode: page table) -> sparse attention (with its log-sum-exp merge).
"""
from __future__ import annotations

import contextlib
import ctypes as C
from typing import Dict, NamedTuple, Optional

import torch

from . import _abi
from ._abi import (MSA_DEVERR_BAD_LEN, MSA_DEVERR_BAD_PAGE, MSA_DEVERR_BAD_ROW, MSA_DEVERR_BAD_SEL,
                   MSA_DEVERR_NO_PAGES, MSA_DEVERR_TIMEOUT, MSA_MODE_CHUNK, MSA_MODE_DECODE, MSA_MODE_PREFILL, MSAError)

__all__ = [
    "msa_index_score", "msa_topk_blocks", "msa_build_page_table", "msa_sparse_attn_prefill",
    "msa_sparse_attn_decode", "msa_sparse_attn_decode_noalloc", "msa_lse_merge", "msa_sparse_attn_prefill_workspace_size",
    "msa_sparse_attn_decode_workspace_size", "msa_cache_append", "decode_step", "prefill_layer", "chunk_layer",
    "msa_dense_attn_decode", "msa_dense_attn_decode_workspace_size", "dense_decode_buffers", "dense_decode_step",
    "msa_dense_attn_prefill", "dense_prefill_layer",
    "msa_plan_step", "msa_release_pages", "plan_buffers", "msa_qk_norm_rope", "Q4Cache", "q4_cache",
    "msa_cache_append_q4", "msa_cache_expand_q4", "msa_attn_decode_q4_workspace_size", "msa_sparse_attn_decode_q4",
    "msa_dense_attn_decode_q4", "decode_q4_buffers", "decode_step_q4",
    "Q8Cache", "q8_cache", "msa_cache_append_q8", "msa_cache_expand_q8", "msa_attn_decode_q8_workspace_size",
    "msa_sparse_attn_decode_q8", "msa_dense_attn_decode_q8", "decode_q8_buffers", "decode_step_q8",
    "msa_window_attn_decode", "msa_window_attn_decode_workspace_size", "msa_window_attn_prefill",
    "msa_fork_requests", "msa_release_shared_pages", "msa_compact_pages", "msa_copy_pages",
    "lib", "MSAError",
    "MSA_MODE_PREFILL", "MSA_MODE_DECODE", "MSA_MODE_CHUNK", "MSA_DEVERR_TIMEOUT", "MSA_DEVERR_BAD_PAGE",
    "MSA_DEVERR_BAD_SEL", "MSA_DEVERR_BAD_LEN", "MSA_DEVERR_NO_PAGES", "MSA_DEVERR_BAD_ROW", "Bk", "D", "dI",
]

Bk = 128
D = 128
dI = 64


def lib():
    return _abi.load()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


def _buffers_on(stream, device):
    """Context of a pipeline's own buffers: torch gives them out, and fills them, in the order of the stream that the calls
    run on (on the current stream, work queued there may still use the memory or fill it later)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _inner_contig(t: torch.Tensor, name: str):
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: innermost dimension must be contiguous")


def _strides(t: torch.Tensor, n: int):
    s = list(t.stride()[:-1])
    return (s + [0] * n)[:n]


# ---------------------------------------------------------------------------
# a1. index score
# ---------------------------------------------------------------------------

def msa_index_score(mode: int, q_idx: torch.Tensor, w: torch.Tensor, k_idx: torch.Tensor, C_out: torch.Tensor,
                    *, seq_pt: Optional[torch.Tensor] = None, seq_len: Optional[torch.Tensor] = None,
                    dev_err: Optional[torch.Tensor] = None, stream=None, k: int = 0,
                    sel: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None,
                    pt: Optional[torch.Tensor] = None, n: Optional[torch.Tensor] = None,
                    last_len: Optional[torch.Tensor] = None, row_scratch: Optional[torch.Tensor] = None,
                    scratch_zeroed: bool = False, q_pos: Optional[torch.Tensor] = None) -> None:
    """Block scores of the Index Branch into ``C_out`` (see msa.h, a1).

    PREFILL: q_idx [B,S,Hkv,HI,dI], w [B,S,Hkv,HI], k_idx [B,S,Hkv,dI], C_out [B,S,Hkv,nb_stride].
    CHUNK:   q_idx, w, C_out as PREFILL; k_idx pool [P,Hkv,Bk,dI], seq_pt [B,max_pages] int32,
             q_pos [B] int32 (position of each sequence's first chunk query).
    DECODE:  q_idx [B,Hkv,HI,dI], w [B,Hkv,HI], k_idx pool [P,Hkv,Bk,dI], C_out [B,Hkv,nb_stride],
             seq_pt [B,max_pages] int32 (contiguous rows), seq_len [B] int32.
    DECODE with ``sel`` given: the same call also selects (a2) into sel/count and,
    with ``pt`` given, builds the page table (a3) into pt/n/last_len; ``row_scratch``
    is B*Hkv int32 of scratch, cleared by the call unless ``scratch_zeroed`` says
    it is already zero (every error-free call leaves it zero).
    """
    for t, nm in ((q_idx, "q_idx"), (w, "w"), (k_idx, "k_idx"), (C_out, "C")):
        _inner_contig(t, nm)
    a = _abi.IndexArgs()
    a.mode = mode
    a.q_idx, a.w, a.k_idx, a.C = _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(C_out)
    a.dev_err = _ptr(dev_err)
    a.nb_stride = C_out.shape[-1]
    if mode in (MSA_MODE_PREFILL, MSA_MODE_CHUNK):
        B, S, Hkv, HI, di = q_idx.shape
        a.B, a.S, a.Hkv, a.HI, a.dI, a.Bk = B, S, Hkv, HI, di, Bk
        a.q_idx_stride[:] = _strides(q_idx, 4)
        a.w_stride[:] = _strides(w, 3)
        a.k_idx_stride[:] = _strides(k_idx, 3)
        a.C_stride[:] = _strides(C_out, 3)
        if mode == MSA_MODE_CHUNK:
            if not (seq_pt.is_contiguous() and q_pos.is_contiguous()):
                raise ValueError("seq_pt and q_pos must be contiguous")
            a.num_pages, a.seq_pt, a.max_pages, a.q_pos = k_idx.shape[0], _ptr(seq_pt), seq_pt.shape[1], _ptr(q_pos)
    else:
        B, Hkv, HI, di = q_idx.shape
        a.B, a.S, a.Hkv, a.HI, a.dI, a.Bk = B, 0, Hkv, HI, di, k_idx.shape[2]
        a.q_idx_stride[:] = _strides(q_idx, 3) + [0]
        a.w_stride[:] = _strides(w, 2) + [0]
        a.k_idx_stride[:] = _strides(k_idx, 3)
        a.C_stride[:] = _strides(C_out, 2) + [0]
        if not seq_pt.is_contiguous():
            raise ValueError("seq_pt must be contiguous")
        a.num_pages = k_idx.shape[0]
        a.seq_pt, a.max_pages, a.seq_len = _ptr(seq_pt), seq_pt.shape[1], _ptr(seq_len)
        if sel is not None:
            for t, nm in ((sel, "sel"), (count, "count"), (row_scratch, "row_scratch")):
                if t is None or not t.is_contiguous():
                    raise ValueError(f"fused selection: {nm} must be a contiguous tensor")
            a.k, a.sel, a.count, a.row_scratch = k, _ptr(sel), _ptr(count), _ptr(row_scratch)
            a.scratch_zeroed = int(bool(scratch_zeroed))
            if pt is not None:
                a.pt, a.n, a.last_len = _ptr(pt), _ptr(n), _ptr(last_len)
    _abi.check(lib().msa_index_score(C.byref(a), _stream(stream)), "msa_index_score")


# ---------------------------------------------------------------------------
# a2. top-k
# ---------------------------------------------------------------------------

def msa_topk_blocks(mode: int, C_in: torch.Tensor, k: int, sel: torch.Tensor, count: torch.Tensor, *,
                    seq_len: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                    stream=None, q_pos: Optional[torch.Tensor] = None) -> None:
    """Own block + top-(k-1) earlier blocks per row (see msa.h, a2).

    PREFILL: C_in [B,S,Hkv,nb], sel [B,S,Hkv,k], count [B,S,Hkv].
    CHUNK:   as PREFILL, own block (q_pos[b] + s) // Bk.
    DECODE:  C_in [B,Hkv,nb], seq_len [B], sel [B,Hkv,k], count [B,Hkv].
    """
    _inner_contig(C_in, "C")
    if not (sel.is_contiguous() and count.is_contiguous()):
        raise ValueError("sel and count must be contiguous")
    a = _abi.TopkArgs()
    a.mode, a.k, a.Bk = mode, k, Bk
    a.C, a.sel, a.count, a.dev_err = _ptr(C_in), _ptr(sel), _ptr(count), _ptr(dev_err)
    a.nb_stride = C_in.shape[-1]
    if mode in (MSA_MODE_PREFILL, MSA_MODE_CHUNK):
        a.B, a.S, a.Hkv = C_in.shape[0], C_in.shape[1], C_in.shape[2]
        a.C_stride[:] = _strides(C_in, 3)
        if mode == MSA_MODE_CHUNK:
            a.q_pos = _ptr(q_pos)
    else:
        a.B, a.S, a.Hkv = C_in.shape[0], 0, C_in.shape[1]
        a.C_stride[:] = _strides(C_in, 2) + [0]
        a.seq_len = _ptr(seq_len)
    _abi.check(lib().msa_topk_blocks(C.byref(a), _stream(stream)), "msa_topk_blocks")


# ---------------------------------------------------------------------------
# a3. page table
# ---------------------------------------------------------------------------

def msa_build_page_table(sel: torch.Tensor, count: torch.Tensor, seq_pt: torch.Tensor, seq_len: torch.Tensor,
                         pt: torch.Tensor, n: torch.Tensor, last_len: torch.Tensor, *,
                         dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Flattened (B*Hkv) page table from the selected blocks (see msa.h, a3)."""
    B, Hkv, k = sel.shape
    for t, nm in ((sel, "sel"), (count, "count"), (pt, "pt"), (n, "n"), (last_len, "last_len")):
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    if not seq_pt.is_contiguous():
        raise ValueError("seq_pt must be contiguous")
    _abi.check(lib().msa_build_page_table(_ptr(sel), _ptr(count), _ptr(seq_pt), seq_pt.shape[1], _ptr(seq_len),
                                          B, Hkv, k, Bk, _ptr(pt), _ptr(n), _ptr(last_len), _ptr(dev_err),
                                          _stream(stream)),
               "msa_build_page_table")


# ---------------------------------------------------------------------------
# a4/a5 sparse attention and a6 merge
# ---------------------------------------------------------------------------

def _prefill_args(Q, K, V, sel, count, O, LSE, softmax_scale, dev_err, seq_pt=None, q_pos=None
                  ) -> _abi.PrefillArgs:
    """PREFILL: K, V [B,S,Hkv,D].  CHUNK (seq_pt and q_pos given): K, V page pools [P,Hkv,Bk,D]."""
    for t, nm in ((Q, "Q"), (K, "K"), (V, "V")):
        _inner_contig(t, nm)
    a = _abi.PrefillArgs()
    a.B, a.S, a.Hq, a.D = Q.shape
    a.Hkv = K.shape[2]
    if seq_pt is not None:
        if not (seq_pt.is_contiguous() and q_pos.is_contiguous()):
            raise ValueError("seq_pt and q_pos must be contiguous")
        a.mode = MSA_MODE_CHUNK
        a.Hkv = K.shape[1]
        a.seq_pt, a.max_pages, a.num_pages, a.q_pos = _ptr(seq_pt), seq_pt.shape[1], K.shape[0], _ptr(q_pos)
    a.Bk = Bk
    a.k = sel.shape[-1]
    a.softmax_scale = softmax_scale
    a.Q, a.K, a.V = _ptr(Q), _ptr(K), _ptr(V)
    a.Q_stride[:] = _strides(Q, 3)
    a.K_stride[:] = _strides(K, 3)
    a.V_stride[:] = _strides(V, 3)
    a.sel, a.count = _ptr(sel), _ptr(count)
    a.O, a.LSE, a.dev_err = _ptr(O), _ptr(LSE), _ptr(dev_err)
    return a


def msa_sparse_attn_prefill_workspace_size(Q, K, sel, chunk_queries: int, max_pages: Optional[int] = None) -> int:
    """Workspace bytes for chunks of ``chunk_queries`` queries; ``max_pages`` (the
    page-table width) selects CHUNK mode, where K is a page pool [P,Hkv,Bk,D]."""
    a = _abi.PrefillArgs()
    a.B, a.S, a.Hq, a.D = Q.shape
    a.Hkv, a.Bk, a.k = K.shape[2], Bk, sel.shape[-1]
    a.Q_stride[:] = _strides(Q, 3)
    a.K_stride[:] = _strides(K, 3)
    a.V_stride[:] = _strides(K, 3)      # V is taken to share K's strides
    if max_pages is not None:
        a.mode, a.Hkv, a.max_pages = MSA_MODE_CHUNK, K.shape[1], int(max_pages)
    return int(lib().msa_sparse_attn_prefill_workspace_size(C.byref(a), int(chunk_queries)))


def msa_sparse_attn_prefill(Q, K, V, sel, count, O, LSE, ws: torch.Tensor, *, softmax_scale: float = 0.0,
                            dev_err=None, stream=None, seq_pt: Optional[torch.Tensor] = None,
                            q_pos: Optional[torch.Tensor] = None) -> None:
    """KV-block-major causal sparse attention (see msa.h, a3'-a4-a6).

    With ``seq_pt`` and ``q_pos`` (CHUNK mode) Q is a chunk of queries at
    positions q_pos[b] + s and K, V are page pools [P,Hkv,Bk,D] indexed by seq_pt."""
    if not (sel.is_contiguous() and count.is_contiguous() and O.is_contiguous()):
        raise ValueError("sel, count and O must be contiguous")
    a = _prefill_args(Q, K, V, sel, count, O, LSE, softmax_scale, dev_err, seq_pt, q_pos)
    _abi.check(lib().msa_sparse_attn_prefill(C.byref(a), _ptr(ws), ws.numel() * ws.element_size(),
                                             _stream(stream)), "msa_sparse_attn_prefill")


def _decode_args(Q, K_pool, V_pool, pt, n, last_len, O, LSE, softmax_scale, dev_err) -> _abi.DecodeArgs:
    for t, nm in ((Q, "Q"), (K_pool, "K_pool"), (V_pool, "V_pool")):
        _inner_contig(t, nm)
    if K_pool.stride() != V_pool.stride():
        raise ValueError("K_pool and V_pool must share strides")
    a = _abi.DecodeArgs()
    a.B, a.Hq, a.D = Q.shape
    a.Hkv, a.Bk = K_pool.shape[1], K_pool.shape[2]
    a.k = pt.shape[-1]
    a.softmax_scale = softmax_scale
    a.Q = _ptr(Q)
    a.Q_stride[:] = _strides(Q, 2)
    a.K_pool, a.V_pool = _ptr(K_pool), _ptr(V_pool)
    a.kv_stride[:] = _strides(K_pool, 3)
    a.num_pages = K_pool.shape[0]
    a.pt, a.n, a.last_len = _ptr(pt), _ptr(n), _ptr(last_len)
    a.O, a.LSE, a.dev_err = _ptr(O), _ptr(LSE), _ptr(dev_err)
    return a


def msa_sparse_attn_decode_workspace_size(B: int, Hq: int, Hkv: int, k: int, D_: int = D) -> int:
    a = _abi.DecodeArgs()
    a.B, a.Hq, a.Hkv, a.k, a.D = B, Hq, Hkv, k, D_
    return int(lib().msa_sparse_attn_decode_workspace_size(C.byref(a)))


def msa_sparse_attn_decode(Q, K_pool, V_pool, pt, n, last_len, O, LSE, ws: torch.Tensor, *,
                           softmax_scale: float = 0.0, dev_err=None, stream=None,
                           scratch_zeroed: bool = False) -> None:
    """Paged sparse attention of one decode step over the flattened page table (see msa.h, a5-a6).

    The workspace's row counters are cleared by the call unless ``scratch_zeroed``
    says they are already zero (every error-free call leaves them zero)."""
    if not (pt.is_contiguous() and n.is_contiguous() and last_len.is_contiguous() and O.is_contiguous()):
        raise ValueError("pt, n, last_len and O must be contiguous")
    a = _decode_args(Q, K_pool, V_pool, pt, n, last_len, O, LSE, softmax_scale, dev_err)
    a.scratch_zeroed = int(bool(scratch_zeroed))
    _abi.check(lib().msa_sparse_attn_decode(C.byref(a), _ptr(ws), ws.numel() * ws.element_size(),
                                            _stream(stream)), "msa_sparse_attn_decode")


def msa_sparse_attn_decode_noalloc(Q, K_pool, V_pool, pt, n, last_len, O, LSE, *, softmax_scale: float = 0.0,
                                   dev_err=None, stream=None) -> None:
    """Same as msa_sparse_attn_decode, for callers that cannot allocate: the
    scratch is the library's built-in device array (see msa.h).  Calls that
    overlap on the GPU share that array and must be serialised."""
    if not (pt.is_contiguous() and n.is_contiguous() and last_len.is_contiguous() and O.is_contiguous()):
        raise ValueError("pt, n, last_len and O must be contiguous")
    a = _decode_args(Q, K_pool, V_pool, pt, n, last_len, O, LSE, softmax_scale, dev_err)
    _abi.check(lib().msa_sparse_attn_decode_noalloc(C.byref(a), _stream(stream)), "msa_sparse_attn_decode_noalloc")


def msa_lse_merge(O_part: torch.Tensor, LSE_part: torch.Tensor, O: torch.Tensor, LSE: Optional[torch.Tensor] = None,
                  *, dev_err=None, stream=None) -> None:
    """O [rows, D] bf16, LSE [rows] from O_part [rows, parts, D] fp32, LSE_part [rows, parts] (see msa.h, a6)."""
    rows, parts, d = O_part.shape
    for t, nm in ((O_part, "O_part"), (LSE_part, "LSE_part"), (O, "O")):
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    _abi.check(lib().msa_lse_merge(_ptr(O_part), _ptr(LSE_part), rows, parts, d, _ptr(O), _ptr(LSE),
                                   _ptr(dev_err), _stream(stream)), "msa_lse_merge")


# ---------------------------------------------------------------------------
# dense comparator (no index branch, no selection)
# ---------------------------------------------------------------------------

def _dense_decode_args(Q, K_pool, V_pool, seq_pt, seq_len, O, LSE, softmax_scale, dev_err) -> _abi.DenseDecodeArgs:
    for t, nm in ((Q, "Q"), (K_pool, "K_pool"), (V_pool, "V_pool")):
        _inner_contig(t, nm)
    if K_pool.stride() != V_pool.stride():
        raise ValueError("K_pool and V_pool must share strides")
    if not seq_pt.is_contiguous():
        raise ValueError("seq_pt must be contiguous")
    a = _abi.DenseDecodeArgs()
    a.B, a.Hq, a.D = Q.shape
    a.Hkv, a.Bk = K_pool.shape[1], K_pool.shape[2]
    a.softmax_scale = softmax_scale
    a.Q = _ptr(Q)
    a.Q_stride[:] = _strides(Q, 2)
    a.K_pool, a.V_pool = _ptr(K_pool), _ptr(V_pool)
    a.kv_stride[:] = _strides(K_pool, 3)
    a.num_pages = K_pool.shape[0]
    a.seq_pt, a.max_pages, a.seq_len = _ptr(seq_pt), seq_pt.shape[1], _ptr(seq_len)
    a.O, a.LSE, a.dev_err = _ptr(O), _ptr(LSE), _ptr(dev_err)
    return a


def msa_dense_attn_decode_workspace_size(B: int, Hq: int, Hkv: int, max_pages: int) -> int:
    a = _abi.DenseDecodeArgs()
    a.B, a.Hq, a.Hkv, a.D, a.Bk, a.max_pages = B, Hq, Hkv, D, Bk, max_pages
    return int(lib().msa_dense_attn_decode_workspace_size(C.byref(a)))


def msa_dense_attn_decode(Q, K_pool, V_pool, seq_pt, seq_len, O, LSE, ws: torch.Tensor, *,
                          softmax_scale: float = 0.0, dev_err=None, stream=None, scratch_zeroed: bool = False) -> None:
    """Dense comparator of a decode step: every cached token of each sequence (see msa.h)."""
    if not O.is_contiguous():
        raise ValueError("O must be contiguous")
    a = _dense_decode_args(Q, K_pool, V_pool, seq_pt, seq_len, O, LSE, softmax_scale, dev_err)
    a.scratch_zeroed = int(bool(scratch_zeroed))
    _abi.check(lib().msa_dense_attn_decode(C.byref(a), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
               "msa_dense_attn_decode")


def dense_decode_buffers(B: int, Hq: int, Hkv: int, max_pages: int, device) -> Dict[str, torch.Tensor]:
    """Outputs and zero-filled scratch of ``dense_decode_step``."""
    dev = torch.device(device)
    return {
        "O": torch.empty(B, Hq, D, dtype=torch.bfloat16, device=dev),
        "LSE": torch.empty(B, Hq, dtype=torch.float32, device=dev),
        "ws": torch.zeros(msa_dense_attn_decode_workspace_size(B, Hq, Hkv, max_pages) // 4 + 64, dtype=torch.float32,
                          device=dev),
        "dev_err": torch.zeros(1, dtype=torch.int32, device=dev),
    }


def dense_decode_step(inp: Dict[str, torch.Tensor], bufs: Optional[Dict[str, torch.Tensor]] = None,
                      softmax_scale: float = 0.0, stream=None, scratch_zeroed: bool = False
                      ) -> Dict[str, torch.Tensor]:
    """The dense comparator of ``decode_step``: attention over every cached token (no index branch)."""
    B, Hq, _ = inp["Q"].shape
    Hkv = inp["K_pool"].shape[1]
    if bufs is None:
        with _buffers_on(stream, inp["Q"].device):
            bufs = dense_decode_buffers(B, Hq, Hkv, inp["seq_pt"].shape[1], inp["Q"].device)
    msa_dense_attn_decode(inp["Q"], inp["K_pool"], inp["V_pool"], inp["seq_pt"], inp["seq_len"], bufs["O"],
                          bufs["LSE"], bufs["ws"], softmax_scale=softmax_scale, dev_err=bufs["dev_err"],
                          stream=stream, scratch_zeroed=scratch_zeroed)
    return bufs


def msa_dense_attn_prefill(Q, K, V, O, LSE, *, softmax_scale: float = 0.0, dev_err=None, stream=None) -> None:
    """Dense comparator of a prefill layer: causal GQA attention over every earlier token (see msa.h).

    Q [B,S,Hq,D], K, V [B,S,Hkv,D] bf16; O [B,S,Hq,D] bf16 and LSE [B,S,Hq] fp32 (dense)."""
    for t, nm in ((Q, "Q"), (K, "K"), (V, "V")):
        _inner_contig(t, nm)
    if not O.is_contiguous() or (LSE is not None and not LSE.is_contiguous()):
        raise ValueError("O and LSE must be contiguous")
    a = _abi.DensePrefillArgs()
    a.B, a.S, a.Hq, a.D = Q.shape
    a.Hkv = K.shape[2]
    a.softmax_scale = softmax_scale
    a.Q, a.K, a.V = _ptr(Q), _ptr(K), _ptr(V)
    a.Q_stride[:] = _strides(Q, 3)
    a.K_stride[:] = _strides(K, 3)
    a.V_stride[:] = _strides(V, 3)
    a.O, a.LSE, a.dev_err = _ptr(O), _ptr(LSE), _ptr(dev_err)
    _abi.check(lib().msa_dense_attn_prefill(C.byref(a), _stream(stream)), "msa_dense_attn_prefill")


def dense_prefill_layer(inp: Dict[str, torch.Tensor], bufs: Optional[Dict[str, torch.Tensor]] = None,
                        softmax_scale: float = 0.0, stream=None) -> Dict[str, torch.Tensor]:
    """The dense comparator of ``prefill_layer``: causal attention over every earlier token (no index branch)."""
    B, S, Hq, _ = inp["Q"].shape
    if bufs is None:
        dev = inp["Q"].device
        with _buffers_on(stream, dev):
            bufs = {"O": torch.empty(B, S, Hq, D, dtype=torch.bfloat16, device=dev),
                    "LSE": torch.empty(B, S, Hq, dtype=torch.float32, device=dev),
                    "dev_err": torch.zeros(1, dtype=torch.int32, device=dev)}
    msa_dense_attn_prefill(inp["Q"], inp["K"], inp["V"], bufs["O"], bufs["LSE"], softmax_scale=softmax_scale,
                           dev_err=bufs["dev_err"], stream=stream)
    return bufs


# ---------------------------------------------------------------------------
# the step before a decode step: append the current tokens to the paged caches
# ---------------------------------------------------------------------------

def msa_cache_append(K_new: torch.Tensor, V_new: torch.Tensor, kidx_new: torch.Tensor, K_pool: torch.Tensor,
                     V_pool: torch.Tensor, kidx_pool: torch.Tensor, seq_pt: torch.Tensor, seq_len: torch.Tensor,
                     *, dev_err=None, stream=None) -> None:
    """Writes token L_b - 1 of every sequence into its page (see msa.h, cache append).

    K_new, V_new [B,Hkv,D], kidx_new [B,Hkv,dI] bf16; K_pool, V_pool [P,Hkv,Bk,D] and
    kidx_pool [P,Hkv,Bk,dI] bf16; seq_pt [B,max_pages] int32 (contiguous rows), seq_len [B].
    With 4-D K_new, V_new [B,T,Hkv,D] and kidx_new [B,T,Hkv,dI] the T tokens of each
    sequence go to positions L_b - T .. L_b - 1.
    """
    for t, nm in ((K_new, "K_new"), (V_new, "V_new"), (kidx_new, "kidx_new"), (K_pool, "K_pool"),
                  (V_pool, "V_pool"), (kidx_pool, "kidx_pool")):
        _inner_contig(t, nm)
    if K_pool.stride() != V_pool.stride():
        raise ValueError("K_pool and V_pool must share strides")
    if not seq_pt.is_contiguous():
        raise ValueError("seq_pt must be contiguous")
    a = _abi.AppendArgs()
    if K_new.dim() == 4:   # several tokens per sequence: strides (b, u, g)
        a.B, a.T, a.Hkv, a.D = K_new.shape
        a.new_t_stride[:] = [K_new.stride(1), V_new.stride(1), kidx_new.stride(1)]
        K_new_bg = [K_new.stride(0), K_new.stride(2)]
        V_new_bg = [V_new.stride(0), V_new.stride(2)]
        X_new_bg = [kidx_new.stride(0), kidx_new.stride(2)]
    else:
        a.B, a.Hkv, a.D = K_new.shape
        a.T = 1
        K_new_bg, V_new_bg, X_new_bg = _strides(K_new, 2), _strides(V_new, 2), _strides(kidx_new, 2)
    a.dI, a.Bk = kidx_new.shape[-1], K_pool.shape[2]
    a.K_new, a.V_new, a.kidx_new = _ptr(K_new), _ptr(V_new), _ptr(kidx_new)
    a.K_new_stride[:] = K_new_bg
    a.V_new_stride[:] = V_new_bg
    a.kidx_new_stride[:] = X_new_bg
    a.K_pool, a.V_pool, a.kidx_pool = _ptr(K_pool), _ptr(V_pool), _ptr(kidx_pool)
    a.kv_stride[:] = _strides(K_pool, 3)
    a.kidx_stride[:] = _strides(kidx_pool, 3)
    a.num_pages = K_pool.shape[0]
    a.seq_pt, a.max_pages, a.seq_len = _ptr(seq_pt), seq_pt.shape[1], _ptr(seq_len)
    a.dev_err = _ptr(dev_err)
    _abi.check(lib().msa_cache_append(C.byref(a), _stream(stream)), "msa_cache_append")


# ---------------------------------------------------------------------------
# the serving step around the cache: page tables and slots, norm with rotation,
# and the cache held in 4 bits.  The tensors are checked and marshalled in
# _msa_binding (csrc/binding.cpp), which raises ValueError where one does not fit.
# ---------------------------------------------------------------------------

def plan_buffers(B: int, N: int, device) -> Dict[str, torch.Tensor]:
    """Outputs of ``msa_plan_step`` for B requests and N token rows."""
    dev = torch.device(device)
    i32 = dict(dtype=torch.int32, device=dev)
    return {"seq_len_out": torch.empty(B, **i32), "free_count_out": torch.empty(1, **i32),
            "cu": torch.empty(B + 1, **i32), "tok_slot": torch.empty(N, dtype=torch.int64, device=dev),
            "tok_pos": torch.empty(N, **i32), "tok_seq": torch.empty(N, **i32)}


def msa_plan_step(seq_len: torch.Tensor, new_len: torch.Tensor, seq_pt: torch.Tensor, free_pages: torch.Tensor,
                  free_count: torch.Tensor, seq_len_out: torch.Tensor, free_count_out: torch.Tensor, cu: torch.Tensor,
                  tok_slot: torch.Tensor, tok_pos: torch.Tensor, tok_seq: Optional[torch.Tensor] = None, *,
                  num_pages: int, dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Pages, positions and slots of the new tokens of every request (see msa.h, page tables and token slots).

    seq_len, new_len [B] int32 (cached and new tokens); seq_pt [B,max_pages] int32, written where pages are given;
    free_pages [F] int32 with free_count [1] int32 (a stack of page ids).  Outputs: seq_len_out [B] (may be seq_len),
    free_count_out [1] (may be free_count), cu [B+1], and for N token rows tok_slot [N] int64, tok_pos and tok_seq [N]
    int32 (-1 in rows past the last token and in those of requests that were not served).  Token rows are packed, in the
    order of the requests; the attention calls take a row per request (its newest token's is cu[b + 1] - 1, if tok_seq
    there is b).
    """
    status = _abi.binding().plan_step(
        seq_len, new_len, seq_pt, free_pages, free_count, seq_len_out, free_count_out, cu, tok_slot, tok_pos, tok_seq,
        num_pages, dev_err, stream)
    if status:
        _abi.check(status, "msa_plan_step")


def msa_release_pages(seq_len: torch.Tensor, done: torch.Tensor, seq_pt: torch.Tensor, free_pages: torch.Tensor,
                      free_count: torch.Tensor, seq_len_out: torch.Tensor, free_count_out: torch.Tensor, *,
                      num_pages: Optional[int] = None, dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Returns the pages of every request with done[b] != 0 to the stack (see msa.h, msa_release_pages).

    seq_len, done [B] int32, seq_pt [B,max_pages] int32 (left as it is), free_pages [F] int32 (written above
    free_count), free_count [1]; seq_len_out [B] and free_count_out [1] may be the inputs.  A page id that goes back and
    is below 0, or at or past ``num_pages`` where that is given, is named in dev_err.
    """
    status = _abi.binding().release_pages(
        seq_len, done, seq_pt, free_pages, free_count, seq_len_out, free_count_out, num_pages, dev_err, stream)
    if status:
        _abi.check(status, "msa_release_pages")


def msa_qk_norm_rope(Q: torch.Tensor, K: Optional[torch.Tensor], pos: torch.Tensor, inv_freq: Optional[torch.Tensor],
                     Q_out: torch.Tensor, K_out: Optional[torch.Tensor], *, V: Optional[torch.Tensor] = None,
                     V_out: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                     q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                     eps: float = 1e-6, interleaved: bool = False, dev_err: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """RMS norm of every query and key head and the position rotation, in one pass (see msa.h).

    Q [N,Hq,D], K and V [N,Hkv,D] bf16 (any token and head strides, innermost contiguous; D = 64 or 128), pos [N] int32,
    inv_freq [rot/2] fp32 (None: no rotation), q_weight and k_weight [D] bf16 or fp32 (None: no norm).  Q_out [N,Hq,D];
    K_out [N,Hkv,D], or with ``slots`` [N] int64 the page pool [P,Hkv,Bk,D] that K goes into, and V into V_out.
    Q_out may be Q and K_out may be K.  Rows with pos < 0 are left out.
    """
    status = _abi.binding().qk_norm_rope(
        Q, K, pos, inv_freq, Q_out, K_out, V, V_out, slots, q_weight, k_weight, eps, interleaved, dev_err, stream)
    if status:
        _abi.check(status, "msa_qk_norm_rope")


class Q4Cache(NamedTuple):
    """A paged K/V cache in 4 bits (see msa.h): codes [P,Hkv,Bk,D/2] and scales [P,Hkv,Bk,D/16], uint8, and one
    power of two for each of K and V."""
    K_codes: torch.Tensor
    K_scales: torch.Tensor
    V_codes: torch.Tensor
    V_scales: torch.Tensor
    k_scale: float = 1.0
    v_scale: float = 1.0


def q4_cache(num_pages: int, Hkv: int, device, k_scale: float = 1.0, v_scale: float = 1.0) -> Q4Cache:
    """A 4-bit cache of zeros."""
    def pool(last):
        return torch.zeros(num_pages, Hkv, Bk, last, dtype=torch.uint8, device=torch.device(device))
    return Q4Cache(pool(D // 2), pool(D // 16), pool(D // 2), pool(D // 16), k_scale, v_scale)


def msa_cache_append_q4(K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, cache: Q4Cache, *,
                        dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Stores K, V [N,Hkv,D] bf16 in 4 bits at slots [N] int64 (page * Bk + row; < 0: not stored) (see msa.h)."""
    status = _abi.binding().cache_append_q4(K, V, slots, cache, dev_err, stream)
    if status:
        _abi.check(status, "msa_cache_append_q4")


def msa_cache_expand_q4(cache: Q4Cache, pages: torch.Tensor, K_out: torch.Tensor, V_out: torch.Tensor, *,
                        dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """The bf16 values of pages [n] int32 into K_out, V_out [n,Hkv,Bk,D] (see msa.h)."""
    status = _abi.binding().cache_expand_q4(cache, pages, K_out, V_out, dev_err, stream)
    if status:
        _abi.check(status, "msa_cache_expand_q4")


def msa_attn_decode_q4_workspace_size(B: int, Hkv: int) -> int:
    return int(lib().msa_attn_decode_q4_workspace_size(B, Hkv))


def msa_sparse_attn_decode_q4(Q: torch.Tensor, cache: Q4Cache, pt: torch.Tensor, n: torch.Tensor,
                              last_len: torch.Tensor, O: torch.Tensor, LSE: Optional[torch.Tensor], ws: torch.Tensor,
                              *, softmax_scale: float = 0.0, dev_err: Optional[torch.Tensor] = None, stream=None,
                              scratch_zeroed: bool = False) -> None:
    """``msa_sparse_attn_decode`` over a 4-bit cache (see msa.h): Q [B,Hq,D] bf16, pt [B*Hkv,k], n, last_len [B*Hkv]
    int32; O [B,Hq,D] bf16, LSE [B,Hq] fp32; ws of ``msa_attn_decode_q4_workspace_size`` bytes."""
    status = _abi.binding().sparse_attn_decode_q4(
        Q, cache, pt, n, last_len, O, LSE, ws, softmax_scale, dev_err, stream, scratch_zeroed)
    if status:
        _abi.check(status, "msa_sparse_attn_decode_q4")


def msa_dense_attn_decode_q4(Q: torch.Tensor, cache: Q4Cache, seq_pt: torch.Tensor, seq_len: torch.Tensor,
                             O: torch.Tensor, LSE: Optional[torch.Tensor], ws: torch.Tensor, *,
                             softmax_scale: float = 0.0, dev_err: Optional[torch.Tensor] = None, stream=None,
                             scratch_zeroed: bool = False) -> None:
    """``msa_dense_attn_decode`` over a 4-bit cache (see msa.h): Q [B,Hq,D] bf16, seq_pt [B,max_pages], seq_len [B]
    int32 (0: an empty sequence); O [B,Hq,D] bf16, LSE [B,Hq] fp32; ws as for ``msa_sparse_attn_decode_q4``."""
    status = _abi.binding().dense_attn_decode_q4(
        Q, cache, seq_pt, seq_len, O, LSE, ws, softmax_scale, dev_err, stream, scratch_zeroed)
    if status:
        _abi.check(status, "msa_dense_attn_decode_q4")


class Q8Cache(NamedTuple):
    """A paged K/V cache in 8 bits (see msa.h): E4M3 codes [P,Hkv,Bk,D] and a scale byte for each page and head [P,Hkv]
    (2^(byte - 127)), uint8."""
    K_codes: torch.Tensor
    K_scales: torch.Tensor
    V_codes: torch.Tensor
    V_scales: torch.Tensor


def q8_cache(num_pages: int, Hkv: int, device) -> Q8Cache:
    """An 8-bit cache of zeros."""
    def pool(*shape):
        return torch.zeros(num_pages, Hkv, *shape, dtype=torch.uint8, device=torch.device(device))
    return Q8Cache(pool(Bk, D), pool(), pool(Bk, D), pool())


def msa_cache_append_q8(K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, cache: Q8Cache, *,
                        dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Stores K, V [N,Hkv,D] bf16 in 8 bits at slots [N] int64 (page * Bk + row; < 0: not stored) (see msa.h).  The tokens
    of a page are consecutive rows in consecutive slots, as ``msa_plan_step`` lays them out; a page fills from row 0 on."""
    status = _abi.binding().cache_append_q8(K, V, slots, cache, dev_err, stream)
    if status:
        _abi.check(status, "msa_cache_append_q8")


def msa_cache_expand_q8(cache: Q8Cache, pages: torch.Tensor, K_out: torch.Tensor, V_out: torch.Tensor, *,
                        dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """The bf16 values of pages [n] int32 into K_out, V_out [n,Hkv,Bk,D] (see msa.h)."""
    status = _abi.binding().cache_expand_q8(cache, pages, K_out, V_out, dev_err, stream)
    if status:
        _abi.check(status, "msa_cache_expand_q8")


def msa_attn_decode_q8_workspace_size(B: int, Hkv: int) -> int:
    return int(lib().msa_attn_decode_q8_workspace_size(B, Hkv))


def msa_sparse_attn_decode_q8(Q: torch.Tensor, cache: Q8Cache, pt: torch.Tensor, n: torch.Tensor,
                              last_len: torch.Tensor, O: torch.Tensor, LSE: Optional[torch.Tensor], ws: torch.Tensor,
                              *, softmax_scale: float = 0.0, dev_err: Optional[torch.Tensor] = None, stream=None,
                              scratch_zeroed: bool = False) -> None:
    """``msa_sparse_attn_decode`` over an 8-bit cache (see msa.h); arguments as in ``msa_sparse_attn_decode_q4``, ws of
    ``msa_attn_decode_q8_workspace_size`` bytes."""
    status = _abi.binding().sparse_attn_decode_q8(
        Q, cache, pt, n, last_len, O, LSE, ws, softmax_scale, dev_err, stream, scratch_zeroed)
    if status:
        _abi.check(status, "msa_sparse_attn_decode_q8")


def msa_dense_attn_decode_q8(Q: torch.Tensor, cache: Q8Cache, seq_pt: torch.Tensor, seq_len: torch.Tensor,
                             O: torch.Tensor, LSE: Optional[torch.Tensor], ws: torch.Tensor, *, window: int = 0,
                             sinks: int = 0, softmax_scale: float = 0.0, dev_err: Optional[torch.Tensor] = None,
                             stream=None, scratch_zeroed: bool = False) -> None:
    """``msa_dense_attn_decode`` over an 8-bit cache (see msa.h): Q [B,Hq,D] bf16, seq_pt [B,max_pages], seq_len [B]
    int32 (0: an empty sequence); O [B,Hq,D] bf16, LSE [B,Hq] fp32; ws as for ``msa_sparse_attn_decode_q8``.  With
    ``window`` > 0 a query sees the last ``window`` tokens and the first ``sinks``."""
    status = _abi.binding().dense_attn_decode_q8(
        Q, cache, seq_pt, seq_len, O, LSE, ws, softmax_scale, dev_err, stream, scratch_zeroed, window, sinks)
    if status:
        _abi.check(status, "msa_dense_attn_decode_q8")


# ---------------------------------------------------------------------------
# pages that several requests hold: forks, their release, compaction, copies
# ---------------------------------------------------------------------------

def msa_fork_requests(src: torch.Tensor, dst: torch.Tensor, seq_len: torch.Tensor, seq_pt: torch.Tensor,
                      free_pages: torch.Tensor, free_count: torch.Tensor, page_shares: torch.Tensor,
                      seq_len_out: torch.Tensor, seq_pt_out: torch.Tensor, free_count_out: torch.Tensor,
                      page_shares_out: torch.Tensor, copy_src: torch.Tensor, copy_dst: torch.Tensor, *,
                      dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Request dst[i] goes on from the cached tokens of request src[i] (see msa.h): full pages are shared, of a page that
    is partly filled the copy is named in copy_src, copy_dst for ``msa_copy_pages``.

    src, dst, copy_src, copy_dst [F] int32 (src < 0: left out); seq_len [B], seq_pt [B,max_pages], free_pages [cap] and
    free_count [1] as in ``msa_plan_step``; page_shares [num_pages] int32, a page's holders beyond the first (0 at the
    start).  The outputs may be the inputs.  How a request is shortened whose pages others hold: msa.h.
    """
    status = _abi.binding().fork_requests(
        src, dst, seq_len, seq_pt, free_pages, free_count, page_shares, seq_len_out, seq_pt_out, free_count_out,
        page_shares_out, copy_src, copy_dst, dev_err, stream)
    if status:
        _abi.check(status, "msa_fork_requests")


def msa_release_shared_pages(seq_len: torch.Tensor, done: torch.Tensor, seq_pt: torch.Tensor, free_pages: torch.Tensor,
                             free_count: torch.Tensor, page_shares: torch.Tensor, seq_len_out: torch.Tensor,
                             free_count_out: torch.Tensor, page_shares_out: torch.Tensor, *,
                             dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """``msa_release_pages`` where requests share pages (see msa.h): a page goes back on the stack with its last holder,
    in the order of page numbers.  seq_len_out, free_count_out and page_shares_out may be the inputs."""
    status = _abi.binding().release_shared_pages(
        seq_len, done, seq_pt, free_pages, free_count, page_shares, seq_len_out, free_count_out, page_shares_out,
        dev_err, stream)
    if status:
        _abi.check(status, "msa_release_shared_pages")


def msa_compact_pages(seq_len: torch.Tensor, seq_pt: torch.Tensor, page_shares: torch.Tensor, seq_pt_out: torch.Tensor,
                      page_shares_out: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor,
                      move_src: torch.Tensor, move_dst: torch.Tensor, *, dev_err: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """The moves (for ``msa_copy_pages``) after which the pages in use are the pool's first ones, the requests' tables
    with the new numbers, and the stack of free pages anew (see msa.h).

    seq_len [B], seq_pt [B,max_pages], page_shares, move_src and move_dst [num_pages] int32; free_pages of at least
    num_pages values and free_count [1] are outputs.  seq_pt_out and page_shares_out may be the inputs.
    """
    status = _abi.binding().compact_pages(
        seq_len, seq_pt, page_shares, seq_pt_out, page_shares_out, free_pages, free_count, move_src, move_dst, dev_err, stream)
    if status:
        _abi.check(status, "msa_compact_pages")


def msa_copy_pages(pools, src: torch.Tensor, dst: torch.Tensor, *, dev_err: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Page src[i] to page dst[i] in every pool (see msa.h): pools a list of up to 16 tensors [P, ..] of any type, each
    page contiguous; src, dst [n] int32, negative ones left out.  No target may be a source or another's target."""
    status = _abi.binding().copy_pages(pools, src, dst, dev_err, stream)
    if status:
        _abi.check(status, "msa_copy_pages")


# ---------------------------------------------------------------------------
# attention through a sliding window with sinks
# ---------------------------------------------------------------------------

def msa_window_attn_decode_workspace_size(B: int, Hkv: int) -> int:
    return int(lib().msa_window_attn_decode_workspace_size(B, Hkv))


def msa_window_attn_decode(Q: torch.Tensor, K_pool: torch.Tensor, V_pool: torch.Tensor, seq_pt: torch.Tensor,
                           seq_len: torch.Tensor, O: torch.Tensor, LSE: Optional[torch.Tensor], ws: torch.Tensor, *,
                           window: int, sinks: int = 0, softmax_scale: float = 0.0,
                           dev_err: Optional[torch.Tensor] = None, stream=None, scratch_zeroed: bool = False) -> None:
    """Decode attention over the last ``window`` tokens of each sequence and its first ``sinks`` (see msa.h): Q [B,Hq,D],
    K_pool, V_pool [P,Hkv,Bk,D] bf16, seq_pt [B,max_pages], seq_len [B] int32 (0: an empty sequence); O [B,Hq,D] bf16,
    LSE [B,Hq] fp32; ws of ``msa_window_attn_decode_workspace_size`` bytes."""
    status = _abi.binding().window_attn_decode(
        Q, K_pool, V_pool, seq_pt, seq_len, O, LSE, ws, softmax_scale, dev_err, stream, scratch_zeroed, window, sinks)
    if status:
        _abi.check(status, "msa_window_attn_decode")


def msa_window_attn_prefill(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
                            LSE: Optional[torch.Tensor], *, window: int, sinks: int = 0,
                            seq_pt: Optional[torch.Tensor] = None, q_pos: Optional[torch.Tensor] = None,
                            softmax_scale: float = 0.0, dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Attention of many queries through a sliding window with sinks (see msa.h): query i sees the tokens t <= i with
    t > i - window or t < sinks.

    Q [B,S,Hq,D]; K, V [B,S,Hkv,D], or with ``seq_pt`` [B,max_pages] and ``q_pos`` [B] int32 the page pools [P,Hkv,Bk,D],
    query s of sequence b then at position q_pos[b] + s (its token in the pages already); all bf16.  O [B,S,Hq,D] bf16 and
    LSE [B,S,Hq] fp32 (dense).  V must be finite for all S (q_pos + S) tokens of a sequence, padding too: a token that a query
    does not see has the weight 0 there, and 0 * inf is NaN.  Slots behind them may hold anything.
    """
    status = _abi.binding().window_attn_prefill(
        Q, K, V, O, LSE, softmax_scale, dev_err, stream, window, sinks, seq_pt, q_pos)
    if status:
        _abi.check(status, "msa_window_attn_prefill")


# ---------------------------------------------------------------------------
# pipelines (hot-path order; marshalling and buffer allocation only)
# ---------------------------------------------------------------------------

def decode_buffers(B: int, Hq: int, Hkv: int, k: int, nb_stride: int, device) -> Dict[str, torch.Tensor]:
    """Output and scratch buffers of one decode step (allocated by torch, owned by the caller).

    The scratch (``ws``, ``row_scratch``) is zero-filled, so calls may pass
    ``scratch_zeroed=True`` from the first one on."""
    dev = torch.device(device)
    return {
        "C": torch.empty(B, Hkv, nb_stride, dtype=torch.float32, device=dev),
        "sel": torch.empty(B, Hkv, k, dtype=torch.int32, device=dev),
        "count": torch.empty(B, Hkv, dtype=torch.int32, device=dev),
        "pt": torch.empty(B * Hkv, k, dtype=torch.int32, device=dev),
        "n": torch.empty(B * Hkv, dtype=torch.int32, device=dev),
        "last_len": torch.empty(B * Hkv, dtype=torch.int32, device=dev),
        "O": torch.empty(B, Hq, D, dtype=torch.bfloat16, device=dev),
        "LSE": torch.empty(B, Hq, dtype=torch.float32, device=dev),
        "ws": torch.zeros(msa_sparse_attn_decode_workspace_size(B, Hq, Hkv, k) // 4 + 64, dtype=torch.float32,
                          device=dev),
        "row_scratch": torch.zeros(B * Hkv, dtype=torch.int32, device=dev),
        "dev_err": torch.zeros(1, dtype=torch.int32, device=dev),
    }


def decode_step(inp: Dict[str, torch.Tensor], k: int, bufs: Optional[Dict[str, torch.Tensor]] = None,
                softmax_scale: float = 0.0, stream=None, fused: bool = True,
                scratch_zeroed: bool = False) -> Dict[str, torch.Tensor]:
    """One MSA decode step: a1 index score -> a2 top-k -> a3 page table -> a5/a6 attention.

    ``inp`` holds Q, q_idx, w, kidx_pool, K_pool, V_pool, seq_pt, seq_len (device tensors; a sequence of length 0 is
    empty: O = 0, LSE = -inf).  With ``fused`` (default) a1-a3 run in one index-score call; otherwise the
    four entry points are called one by one.  ``scratch_zeroed`` skips the
    counter clears (valid with ``decode_buffers`` scratch that every previous
    call left zero, i.e. no device error was raised).
    """
    B, Hq, _ = inp["Q"].shape
    Hkv = inp["K_pool"].shape[1]
    if bufs is None:
        with _buffers_on(stream, inp["Q"].device):
            bufs = decode_buffers(B, Hq, Hkv, k, inp["seq_pt"].shape[1], inp["Q"].device)
    e = bufs["dev_err"]
    if fused:
        msa_index_score(MSA_MODE_DECODE, inp["q_idx"], inp["w"], inp["kidx_pool"], bufs["C"], seq_pt=inp["seq_pt"],
                        seq_len=inp["seq_len"], dev_err=e, stream=stream, k=k, sel=bufs["sel"],
                        count=bufs["count"], pt=bufs["pt"], n=bufs["n"], last_len=bufs["last_len"],
                        row_scratch=bufs["row_scratch"], scratch_zeroed=scratch_zeroed)
    else:
        msa_index_score(MSA_MODE_DECODE, inp["q_idx"], inp["w"], inp["kidx_pool"], bufs["C"], seq_pt=inp["seq_pt"],
                        seq_len=inp["seq_len"], dev_err=e, stream=stream)
        msa_topk_blocks(MSA_MODE_DECODE, bufs["C"], k, bufs["sel"], bufs["count"], seq_len=inp["seq_len"],
                        dev_err=e, stream=stream)
        msa_build_page_table(bufs["sel"], bufs["count"], inp["seq_pt"], inp["seq_len"], bufs["pt"], bufs["n"],
                             bufs["last_len"], dev_err=e, stream=stream)
    msa_sparse_attn_decode(inp["Q"], inp["K_pool"], inp["V_pool"], bufs["pt"], bufs["n"], bufs["last_len"],
                           bufs["O"], bufs["LSE"], bufs["ws"], softmax_scale=softmax_scale, dev_err=e,
                           stream=stream, scratch_zeroed=scratch_zeroed)
    return bufs


def decode_q4_buffers(B: int, Hq: int, Hkv: int, k: int, nb_stride: int, device) -> Dict[str, torch.Tensor]:
    """``decode_buffers`` with the workspace of the 4-bit attention."""
    dev = torch.device(device)
    bufs = {n: t for n, t in decode_buffers(B, Hq, Hkv, k, nb_stride, dev).items() if n != "ws"}
    bufs["ws"] = torch.zeros(msa_attn_decode_q4_workspace_size(B, Hkv), dtype=torch.uint8, device=dev)
    return bufs


def _decode_step_paged(inp, Hkv, k, bufs, softmax_scale, stream, scratch_zeroed, buffers, attend):
    """Index score, selection and page table, then ``attend`` over the selected pages of a cache."""
    dev = inp["Q"].device
    if dev.type == "cuda" and dev.index != torch.cuda.current_device():   # the index call would go to the current one
        with torch.cuda.device(dev):
            return _decode_step_paged(inp, Hkv, k, bufs, softmax_scale, stream, scratch_zeroed, buffers, attend)
    B, Hq, _ = inp["Q"].shape
    if bufs is None:
        with _buffers_on(stream, dev):
            bufs = buffers(B, Hq, Hkv, k, inp["seq_pt"].shape[1], dev)
    e = bufs["dev_err"]
    msa_index_score(MSA_MODE_DECODE, inp["q_idx"], inp["w"], inp["kidx_pool"], bufs["C"], seq_pt=inp["seq_pt"],
                    seq_len=inp["seq_len"], dev_err=e, stream=stream, k=k, sel=bufs["sel"], count=bufs["count"],
                    pt=bufs["pt"], n=bufs["n"], last_len=bufs["last_len"], row_scratch=bufs["row_scratch"],
                    scratch_zeroed=scratch_zeroed)
    attend(inp["Q"], bufs["pt"], bufs["n"], bufs["last_len"], bufs["O"], bufs["LSE"], bufs["ws"],
           softmax_scale=softmax_scale, dev_err=e, stream=stream, scratch_zeroed=scratch_zeroed)
    return bufs


def decode_step_q4(inp: Dict[str, torch.Tensor], cache: Q4Cache, k: int,
                   bufs: Optional[Dict[str, torch.Tensor]] = None, softmax_scale: float = 0.0, stream=None,
                   scratch_zeroed: bool = False) -> Dict[str, torch.Tensor]:
    """``decode_step`` with K and V in a 4-bit cache: the index branch and selection are the same (``inp`` holds Q,
    q_idx, w, kidx_pool, seq_pt, seq_len), the attention reads ``cache``.  Row b of Q, q_idx and w is sequence b's
    query; a sequence of length 0 is empty (O = 0, LSE = -inf).  The step runs on the tensors' device."""
    def attend(Q, *rest, **kw):
        msa_sparse_attn_decode_q4(Q, cache, *rest, **kw)
    return _decode_step_paged(inp, cache.K_codes.shape[1], k, bufs, softmax_scale, stream, scratch_zeroed,
                              decode_q4_buffers, attend)


def decode_q8_buffers(B: int, Hq: int, Hkv: int, k: int, nb_stride: int, device) -> Dict[str, torch.Tensor]:
    """``decode_buffers`` with the workspace of the 8-bit attention."""
    dev = torch.device(device)
    bufs = {n: t for n, t in decode_buffers(B, Hq, Hkv, k, nb_stride, dev).items() if n != "ws"}
    bufs["ws"] = torch.zeros(msa_attn_decode_q8_workspace_size(B, Hkv), dtype=torch.uint8, device=dev)
    return bufs


def decode_step_q8(inp: Dict[str, torch.Tensor], cache: Q8Cache, k: int,
                   bufs: Optional[Dict[str, torch.Tensor]] = None, softmax_scale: float = 0.0, stream=None,
                   scratch_zeroed: bool = False) -> Dict[str, torch.Tensor]:
    """``decode_step`` with K and V in an 8-bit cache: the index branch and selection are the same (``inp`` holds Q,
    q_idx, w, kidx_pool, seq_pt, seq_len), the attention reads ``cache``.  Row b of Q, q_idx and w is sequence b's
    query; a sequence of length 0 is empty (O = 0, LSE = -inf).  The step runs on the tensors' device."""
    def attend(Q, *rest, **kw):
        msa_sparse_attn_decode_q8(Q, cache, *rest, **kw)
    return _decode_step_paged(inp, cache.K_codes.shape[1], k, bufs, softmax_scale, stream, scratch_zeroed,
                              decode_q8_buffers, attend)


def prefill_buffers(B: int, S: int, Hq: int, Hkv: int, k: int, device, ws_bytes: int) -> Dict[str, torch.Tensor]:
    dev = torch.device(device)
    nb = (S + Bk - 1) // Bk
    return {
        "C": torch.empty(B, S, Hkv, nb, dtype=torch.float32, device=dev),
        "sel": torch.empty(B, S, Hkv, k, dtype=torch.int32, device=dev),
        "count": torch.empty(B, S, Hkv, dtype=torch.int32, device=dev),
        "O": torch.empty(B, S, Hq, D, dtype=torch.bfloat16, device=dev),
        "LSE": torch.empty(B, S, Hq, dtype=torch.float32, device=dev),
        "ws": torch.empty((ws_bytes + 15) // 16 * 4, dtype=torch.float32, device=dev),
        "dev_err": torch.zeros(1, dtype=torch.int32, device=dev),
    }


def prefill_layer(inp: Dict[str, torch.Tensor], k: int, bufs: Optional[Dict[str, torch.Tensor]] = None,
                  ws_bytes: Optional[int] = None, softmax_scale: float = 0.0, stream=None
                  ) -> Dict[str, torch.Tensor]:
    """One MSA prefill layer: a1 index score -> a2 top-k -> a3'/a4/a6 KV-block-major attention.

    ``inp`` holds Q, K, V, q_idx, k_idx, w (device tensors).
    """
    B, S, Hq, _ = inp["Q"].shape
    Hkv = inp["K"].shape[2]
    if bufs is None:
        if ws_bytes is None:
            sel_probe = torch.empty(1, 1, 1, k, dtype=torch.int32)
            ws_bytes = msa_sparse_attn_prefill_workspace_size(inp["Q"], inp["K"], sel_probe, min(S, 8192) * B)
        with _buffers_on(stream, inp["Q"].device):
            bufs = prefill_buffers(B, S, Hq, Hkv, k, inp["Q"].device, ws_bytes)
    e = bufs["dev_err"]
    msa_index_score(MSA_MODE_PREFILL, inp["q_idx"], inp["w"], inp["k_idx"], bufs["C"], dev_err=e, stream=stream)
    msa_topk_blocks(MSA_MODE_PREFILL, bufs["C"], k, bufs["sel"], bufs["count"], dev_err=e, stream=stream)
    msa_sparse_attn_prefill(inp["Q"], inp["K"], inp["V"], bufs["sel"], bufs["count"], bufs["O"], bufs["LSE"],
                            bufs["ws"], softmax_scale=softmax_scale, dev_err=e, stream=stream)
    return bufs


def chunk_buffers(B: int, S: int, Hq: int, Hkv: int, k: int, nb: int, device, ws_bytes: int
                  ) -> Dict[str, torch.Tensor]:
    """Outputs and scratch of ``chunk_layer`` (score rows of ``nb`` blocks)."""
    bufs = prefill_buffers(B, S, Hq, Hkv, k, device, ws_bytes)
    bufs["C"] = torch.empty(B, S, Hkv, nb, dtype=torch.float32, device=torch.device(device))
    return bufs


def chunk_layer(inp: Dict[str, torch.Tensor], k: int, bufs: Optional[Dict[str, torch.Tensor]] = None,
                ws_bytes: Optional[int] = None, softmax_scale: float = 0.0, stream=None
                ) -> Dict[str, torch.Tensor]:
    """One MSA layer over a chunk of S queries per sequence on a paged cache
    (chunked prefill over a cached prefix, or several decode tokens per
    sequence): a1 index score -> a2 top-k -> a3'/a4/a6 KV-block-major attention.

    ``inp`` holds Q [B,S,Hq,D], q_idx [B,S,Hkv,HI,dI], w [B,S,Hkv,HI], the page
    pools K_pool, V_pool [P,Hkv,Bk,D] and kidx_pool [P,Hkv,Bk,dI], seq_pt
    [B,max_pages] and q_pos [B] int32 (the chunk's own tokens already in the
    pages).  Score rows span max_pages blocks unless ``bufs`` says otherwise.
    With ``kv_seq_pt`` [B,max_pages] in ``inp`` K_pool and V_pool have a page table of
    their own: the expanded pages of a 4-bit cache (``msa_cache_expand_q4``), beside
    index keys in the cache's pages.
    """
    B, S, Hq, _ = inp["Q"].shape
    Hkv = inp["K_pool"].shape[1]
    max_pages = inp["seq_pt"].shape[1]
    kv_pt = inp.get("kv_seq_pt", inp["seq_pt"])
    if bufs is None:
        if ws_bytes is None:
            sel_probe = torch.empty(1, 1, 1, k, dtype=torch.int32)
            ws_bytes = msa_sparse_attn_prefill_workspace_size(inp["Q"], inp["K_pool"], sel_probe,
                                                              min(S, 8192) * B, max_pages=kv_pt.shape[1])
        with _buffers_on(stream, inp["Q"].device):
            bufs = chunk_buffers(B, S, Hq, Hkv, k, max_pages, inp["Q"].device, ws_bytes)
    e = bufs["dev_err"]
    msa_index_score(MSA_MODE_CHUNK, inp["q_idx"], inp["w"], inp["kidx_pool"], bufs["C"], seq_pt=inp["seq_pt"],
                    q_pos=inp["q_pos"], dev_err=e, stream=stream)
    msa_topk_blocks(MSA_MODE_CHUNK, bufs["C"], k, bufs["sel"], bufs["count"], q_pos=inp["q_pos"], dev_err=e,
                    stream=stream)
    msa_sparse_attn_prefill(inp["Q"], inp["K_pool"], inp["V_pool"], bufs["sel"], bufs["count"], bufs["O"],
                            bufs["LSE"], bufs["ws"], softmax_scale=softmax_scale, dev_err=e, stream=stream,
                            seq_pt=kv_pt, q_pos=inp["q_pos"])
    return bufs
