"""ctypes binding of ``libdsa.so`` (C ABI in ``include/dsa.h``).

Argument marshalling only: each function checks dtypes and shapes of the
torch tensors it is given, passes their device pointers and the current CUDA
stream to the C entry point of the same name, and raises ``DSAError`` on a
non-zero status.  Every arithmetic step runs in the library's CUDA kernels;
there is no other implementation behind these names, and a missing library
raises instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")
PAGE_SIZE = 64

_lib = None


class DSAError(RuntimeError):
    pass


_P, _I, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float

_SIGNATURES = {
    "dsa_status_string": ([_I], ctypes.c_char_p),
    "dsa_version": ([], _I),
    "dsa_last_error_string": ([], ctypes.c_char_p),
    "dsa_check_device_error": ([], _I),
    "dsa_set_wait_limit_ns": ([ctypes.c_ulonglong], _I),
    "dsa_row_stats_bytes": ([_I], _SZ),
    "dsa_indexer_scores": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I64, _P, _P], _I),
    "dsa_topk_workspace_size": ([_I, _I, _I], _SZ),
    "dsa_topk": ([_P, _I64, _I, _I, _P, _I, _I, _P, _P, _P, _SZ, _P], _I),
    "dsa_indexer_topk_workspace_size": ([_I, _I, _I, _I, _I], _SZ),
    "dsa_indexer_topk": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P, _P], _I),
    "dsa_indexer_topk_varlen": ([_P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _I, _I, _P, _P, _SZ, _P, _P], _I),
    "dsa_sparse_gqa_prefill_varlen": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P], _I),
    "dsa_indexer_topk_threshold": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P, _P], _I),
    "dsa_indexer_topk_candidates": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P, _P], _I),
    "dsa_indexer_topk_select": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P, _P], _I),
    "dsa_indexer_kl": ([_P, _I64, _I, _I, _P, _I, _I64, _P, _I, _P, _P, _P], _I),
    "dsa_sparse_gqa_prefill": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P], _I),
    "dsa_decode_workspace_size": ([_I, _I, _I, _I, _I, _I], _SZ),
    "dsa_sparse_gqa_decode": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _I,
                               _I, _I, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P, _P], _I),
    "dsa_decode_indexer_scores": ([_P, _P, _P, _P, _P, _P, _I, _I, _P, _I, _I, _I, _I, _P, _I64, _P], _I),
    "dsa_decode_attention_workspace_size": ([_I, _I, _I, _I, _I], _SZ),
    "dsa_sparse_gqa_decode_attention": ([_P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _F,
                                         _P, _SZ, _P, _P, _P], _I),
    "dsa_decode_attention_fixed_scratch_bytes": ([], _SZ),
    "dsa_sparse_gqa_decode_attention_noalloc": ([_P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _F,
                                                 _P, _P, _P], _I),
    "dsa_kv8_append": ([_P, _I64, _P, _I64, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _I,
                        _P, _P, _P, _P, _P, _P], _I),
    "dsa_sparse_gqa_decode_attention_kv8": ([_P, _P, _P, _P, _I, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _F,
                                             _P, _P, _P], _I),
    "dsa_sparse_gqa_prefill_kv8": ([_P, _P, _P, _P, _I, _P, _I, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                                    _P, _P, _P], _I),
    "dsa_decode_kv8_workspace_size": ([_I, _I, _I], _SZ),
    "dsa_sparse_gqa_decode_kv8": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _P, _I,
                                   _I, _I, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P, _P], _I),
    "dsa_pages_extend": ([_P, _P, _I, _P, _I, _I, _P, _P, _I, _P, _P], _I),
    "dsa_pages_fork": ([_P, _P, _I, _P, _P, _I, _P, _I, _I, _P, _P, _I, _P, _P], _I),
    "dsa_pages_free": ([_P, _I, _P, _I, _I, _P, _P, _I, _P], _I),
    "dsa_pages_copy": ([_P, _P, _I, _P, _P, _I, _I, _P], _I),
    "dsa_pages_compact_workspace_size": ([_I], _SZ),
    "dsa_pages_compact": ([_P, _P, _I, _P, _P, _I, _I, _P, _P, _P, _I, _P, _P, _P, _SZ, _P], _I),
    "dsa_read_probe": ([_P, _SZ, _I, _P, _P], _I),
}


def lib():
    """Open libdsa.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise DSAError(f"{LIB_PATH} is missing; build it with `python -m sparse_long_context_03_b200.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def exported_symbols():
    return list(_SIGNATURES)


def version() -> int:
    return lib().dsa_version()


def status_string(code: int) -> str:
    return lib().dsa_status_string(int(code)).decode()


def check_device_error():
    """Synchronises; raises DSAError if a kernel's bounded wait expired."""
    _check(lib().dsa_check_device_error(), "dsa_check_device_error")


def device_error_status() -> int:
    """dsa_check_device_error's status code (0 = none), without raising."""
    return int(lib().dsa_check_device_error())


def set_wait_limit_ns(ns: int) -> None:
    """dsa_set_wait_limit_ns: bound of the prefill indexer's pipeline waits
    on the current device (0 restores the default).  For failure-path tests."""
    _check(lib().dsa_set_wait_limit_ns(int(ns)), "dsa_set_wait_limit_ns")


def _check(code: int, name: str):
    if code != 0:
        err = lib().dsa_last_error_string().decode()
        raise DSAError(f"{name}: {status_string(code)}" + (f" ({err})" if err else ""))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _need(t, dtype, ndim, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")


# ---------------------------------------------------------------------------
# prefill
# ---------------------------------------------------------------------------

def row_stats_bytes(n_rows) -> int:
    return int(lib().dsa_row_stats_bytes(int(n_rows)))


def indexer_scores(q8, q_scale, w, k8, k_scale, row_begin, n_rows, scores, row_stats=None, stream=None):
    """dsa_indexer_scores: rows [row_begin, row_begin+n_rows) of the causal
    lightning-indexer score matrix into ``scores`` [n_rows, ld] float32;
    optionally the rows' value ranges into ``row_stats`` for dsa_topk."""
    _need(q8, torch.uint8, 3, "q8")
    _need(k8, torch.uint8, 2, "k8")
    _need(scores, torch.float32, 2, "scores")
    L, HI, dI = q8.shape
    _check(lib().dsa_indexer_scores(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8), _ptr(k_scale), L, HI, dI,
                                    int(row_begin), int(n_rows), _ptr(scores), scores.stride(0), _ptr(row_stats),
                                    _stream(stream)),
           "dsa_indexer_scores")


def topk_workspace_size(n_rows, max_len, k) -> int:
    return int(lib().dsa_topk_workspace_size(int(n_rows), int(max_len), int(k)))


def topk(scores, row_begin, n_rows, k, idx, row_len=None, max_len=None, ws=None, row_stats=None, stream=None):
    """dsa_topk: per-row top-k (ascending indices, -1 padded) into idx [n_rows, k]."""
    _need(scores, torch.float32, 2, "scores")
    _need(idx, torch.int32, 2, "idx")
    if max_len is None:
        max_len = scores.shape[1] if row_len is not None else row_begin + n_rows
    need = topk_workspace_size(n_rows, max_len, k)
    ws_bytes = 0
    if need:
        if ws is None:
            raise DSAError(f"dsa_topk needs a {need}-byte workspace")
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().dsa_topk(_ptr(scores), scores.stride(0), int(row_begin), int(n_rows), _ptr(row_len), int(max_len),
                          int(k), _ptr(idx), _ptr(row_stats), _ptr(ws), ws_bytes, _stream(stream)), "dsa_topk")


def indexer_topk_workspace_size(row_begin, n_rows, k, HI, dI) -> int:
    return int(lib().dsa_indexer_topk_workspace_size(int(row_begin), int(n_rows), int(k), int(HI), int(dI)))


_TOPK_STAGES = {None: "dsa_indexer_topk", "threshold": "dsa_indexer_topk_threshold",
                "candidates": "dsa_indexer_topk_candidates", "select": "dsa_indexer_topk_select"}


def indexer_topk(q8, q_scale, w, k8, k_scale, row_begin, n_rows, k, idx, ws, stats=None, stream=None,
                 stage=None):
    """dsa_indexer_topk: Omega_t of query rows [row_begin, row_begin+n_rows)
    (the top-k of their causal indexer scores, ascending, -1 padded) into
    idx [n_rows, k] int32, without writing the score matrix.  ``ws`` is a
    uint8 CUDA tensor of indexer_topk_workspace_size(...) bytes or more;
    ``stats`` (optional int64 CUDA tensor of 2) receives the number of rows
    scored again in full and the number of candidates kept.  ``stage`` = "threshold", "candidates" or "select"
    runs one stage only (dsa_indexer_topk_<stage>)."""
    _need(q8, torch.uint8, 3, "q8")
    _need(k8, torch.uint8, 2, "k8")
    _need(idx, torch.int32, 2, "idx")
    name = _TOPK_STAGES[stage]
    L, HI, dI = q8.shape
    _check(getattr(lib(), name)(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8), _ptr(k_scale), L, HI, dI,
                                int(row_begin), int(n_rows), int(k), _ptr(idx), _ptr(ws),
                                ws.numel() * ws.element_size(), _ptr(stats), _stream(stream)), name)


def indexer_kl(scores, row_begin, n_rows, p, loss_rows, idx=None, loss_total=None, stream=None):
    """dsa_indexer_kl: per-row indexer distillation loss
    sum_g KL(p[r,g,S] normalised || Softmax(I[t,S])) into loss_rows [n_rows]
    float64; S = [0, t] (idx None: dense warm-up) or the valid entries of idx
    row r (sparse adaptation).  scores [n_rows, ld] float32, p [n_rows, G,
    ld_p] float32; loss_total (optional, 1 float64) gets the sum."""
    _need(scores, torch.float32, 2, "scores")
    _need(p, torch.float32, 3, "p")
    _need(loss_rows, torch.float64, 1, "loss_rows")
    k = 0
    if idx is not None:
        _need(idx, torch.int32, 2, "idx")
        k = idx.shape[1]
    _check(lib().dsa_indexer_kl(_ptr(scores), scores.stride(0), int(row_begin), int(n_rows), _ptr(p), p.shape[1],
                                p.stride(1), _ptr(idx), k, _ptr(loss_rows), _ptr(loss_total), _stream(stream)),
           "dsa_indexer_kl")


def sparse_gqa_prefill(Q, K, V, idx, row_begin, n_rows, k, sm_scale, O, lse=None, stream=None):
    """dsa_sparse_gqa_prefill: attention of query rows [row_begin, row_begin+n_rows)
    over their selected keys.  Q/O [n_rows,Hq,D] bf16, K/V [L,Hkv,D] bf16."""
    for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (O, "O")):
        _need(t, torch.bfloat16, 3, n)
    _need(idx, torch.int32, 2, "idx")
    Hq, D = Q.shape[1], Q.shape[2]
    Hkv = K.shape[1]
    _check(lib().dsa_sparse_gqa_prefill(_ptr(Q), _ptr(K), _ptr(V), _ptr(idx), int(row_begin), int(n_rows), Hq, Hkv,
                                        D, int(k), float(sm_scale), _ptr(O), _ptr(lse), _stream(stream)),
           "dsa_sparse_gqa_prefill")


def indexer_topk_varlen(q8, q_scale, w, k8, k_scale, cu_seqlens, row_begin, n_rows, k, idx, ws, stats=None,
                        stream=None):
    """dsa_indexer_topk_varlen: Omega_t of packed query rows [row_begin,
    row_begin+n_rows); cu_seqlens int32 CUDA tensor [nseq+1].  idx [n_rows,
    k] receives positions within each query's own sequence."""
    _need(q8, torch.uint8, 3, "q8")
    _need(k8, torch.uint8, 2, "k8")
    _need(idx, torch.int32, 2, "idx")
    _need(cu_seqlens, torch.int32, 1, "cu_seqlens")
    L, HI, dI = q8.shape
    _check(lib().dsa_indexer_topk_varlen(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8), _ptr(k_scale), L, HI, dI,
                                         _ptr(cu_seqlens), cu_seqlens.numel() - 1, int(row_begin), int(n_rows), int(k),
                                         _ptr(idx), _ptr(ws), ws.numel() * ws.element_size(), _ptr(stats),
                                         _stream(stream)), "dsa_indexer_topk_varlen")


def sparse_gqa_prefill_varlen(Q, K, V, idx, cu_seqlens, row_begin, n_rows, k, sm_scale, O, lse=None, stream=None):
    """dsa_sparse_gqa_prefill_varlen: attention of packed query rows over
    their selected positions (relative to each query's own sequence)."""
    for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (O, "O")):
        _need(t, torch.bfloat16, 3, n)
    _need(idx, torch.int32, 2, "idx")
    _need(cu_seqlens, torch.int32, 1, "cu_seqlens")
    Hq, D = Q.shape[1], Q.shape[2]
    Hkv = K.shape[1]
    _check(lib().dsa_sparse_gqa_prefill_varlen(_ptr(Q), _ptr(K), _ptr(V), _ptr(idx), _ptr(cu_seqlens),
                                               cu_seqlens.numel() - 1, int(row_begin), int(n_rows), Hq, Hkv, D,
                                               int(k), float(sm_scale), _ptr(O), _ptr(lse), _stream(stream)),
           "dsa_sparse_gqa_prefill_varlen")


class PrefillPlan:
    """Buffers for a prefill of one sequence.

    fused=True (the default where the shape allows it): the fused indexer +
    top-k (dsa_indexer_topk), whose workspace holds sampled scores,
    thresholds and candidate lists instead of the score matrix; query rows
    are chunked only to keep that workspace within ``fused_budget_bytes``.
    fused=False: the score matrix of one chunk of query rows at a time
    ([chunk_rows, ld] float32, the chunked indexer of report section 5.2.1),
    then dsa_topk."""

    def __init__(self, L, HI, dI, Hq, Hkv, D, k, chunk_rows=None, device="cuda", score_budget_bytes=4 << 30,
                 fused=None, fused_budget_bytes=24 << 30):
        self.L, self.HI, self.dI, self.Hq, self.Hkv, self.D, self.k = L, HI, dI, Hq, Hkv, D, k
        self.ld = (L + 3) // 4 * 4
        if fused is None:
            fused = indexer_topk_workspace_size(0, 1, k, HI, dI) > 0
        self.fused = bool(fused)
        self.idx = torch.empty(L, k, dtype=torch.int32, device=device)
        if self.fused:
            if chunk_rows is None:
                chunk_rows = L
                while chunk_rows > 1 and self._fused_ws(chunk_rows) > fused_budget_bytes:
                    chunk_rows = (chunk_rows + 1) // 2
            self.chunk_rows = int(chunk_rows)
            self.scores = None
            self.row_stats = None
            self.ws = torch.empty(max(self._fused_ws(self.chunk_rows), 1), dtype=torch.uint8, device=device)
            self.stats = torch.zeros(2, dtype=torch.int64, device=device)
        else:
            if chunk_rows is None:
                chunk_rows = max(1, min(L, score_budget_bytes // (4 * self.ld)))
            self.chunk_rows = int(chunk_rows)
            self.scores = torch.empty(self.chunk_rows, self.ld, dtype=torch.float32, device=device)
            need = topk_workspace_size(self.chunk_rows, L, k)
            self.ws = torch.empty(max(need, 1), dtype=torch.uint8, device=device) if need else None
            self.row_stats = torch.empty(row_stats_bytes(self.chunk_rows), dtype=torch.uint8, device=device)
            self.stats = None

    def _fused_ws(self, chunk_rows):
        # the workspace grows with the chunk's last row, so the last chunk needs the most
        need = 0
        for r0 in range(0, self.L, chunk_rows):
            need = max(need, indexer_topk_workspace_size(r0, min(chunk_rows, self.L - r0), self.k, self.HI, self.dI))
        return need

    def chunks(self):
        for r0 in range(0, self.L, self.chunk_rows):
            yield r0, min(self.chunk_rows, self.L - r0)


def select_rows(plan: PrefillPlan, q8, sq, w, k8, sk, stream=None):
    """Omega_t of every query row into plan.idx [L, k]: the fused indexer +
    top-k, or the chunked score matrix followed by dsa_topk."""
    for r0, n in plan.chunks():
        if plan.fused:
            indexer_topk(q8, sq, w, k8, sk, r0, n, plan.k, plan.idx[r0:r0 + n], plan.ws, stream=stream)
        else:
            indexer_scores(q8, sq, w, k8, sk, r0, n, plan.scores[:n], row_stats=plan.row_stats, stream=stream)
            topk(plan.scores[:n], r0, n, plan.k, plan.idx[r0:r0 + n], max_len=r0 + n, ws=plan.ws,
                 row_stats=plan.row_stats, stream=stream)


def prefill_forward(plan: PrefillPlan, q8, sq, w, k8, sk, Q, K, V, O, sm_scale=None, lse=None, stream=None):
    """Whole DSA prefill of one sequence: Omega_t of every query row (the
    indexer and the top-k), then the sparse attention of every row.
    Writes plan.idx [L,k] and O [L,Hq,D] (lse [L,Hq] if given)."""
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(plan.D)
    select_rows(plan, q8, sq, w, k8, sk, stream=stream)
    sparse_gqa_prefill(Q, K, V, plan.idx, 0, plan.L, plan.k, sm_scale, O, lse, stream=stream)


def prefill_forward_packed(plan: PrefillPlan, cu_seqlens, q8, sq, w, k8, sk, Q, K, V, O, sm_scale=None, lse=None,
                           idx_out=None, stream=None):
    """DSA prefill of several sequences packed along the token axis: sequence
    b holds tokens cu_seqlens[b] .. cu_seqlens[b+1]-1 and is its own causal
    prefill -- no query scores or attends a key of another sequence.  Every
    per-token tensor (q8, sq, w, k8, sk, Q, K, V, O, lse) is indexed by the
    packed token.  idx_out, if given, [total, k] int32, receives each token's
    selected positions within its own sequence.

    With the fused indexer + top-k (plan.fused; the plan sized for the
    packed total), every stage is one launch per chunk of packed rows over
    all sequences at once (dsa_indexer_topk_varlen,
    dsa_sparse_gqa_prefill_varlen; cu_seqlens as a host sequence or an int32
    CUDA tensor).  Otherwise (HI = 4) the score-matrix chain runs once per
    sequence on its slice (cu_seqlens host ints; the plan sized for the
    longest sequence)."""
    cu = [int(x) for x in (cu_seqlens.tolist() if isinstance(cu_seqlens, torch.Tensor) else cu_seqlens)]
    if any(b < a for a, b in zip(cu, cu[1:])) or (cu and cu[0] != 0):
        raise DSAError("cu_seqlens must start at 0 and be non-decreasing")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(plan.D)
    total = cu[-1] if cu else 0
    if plan.fused:
        if total > plan.L:
            raise DSAError("the packed tokens exceed the plan")
        cu_dev = cu_seqlens if isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.is_cuda else \
            torch.tensor(cu, dtype=torch.int32, device=q8.device)
        idx = plan.idx[:total] if idx_out is None else idx_out
        for r0 in range(0, total, plan.chunk_rows):
            n = min(plan.chunk_rows, total - r0)
            indexer_topk_varlen(q8, sq, w, k8, sk, cu_dev, r0, n, plan.k, idx[r0:r0 + n], plan.ws, stream=stream)
        sparse_gqa_prefill_varlen(Q, K, V, idx, cu_dev, 0, total, plan.k, sm_scale, O, lse, stream=stream)
        return
    if max((b - a for a, b in zip(cu, cu[1:])), default=0) > plan.L:
        raise DSAError("a sequence is longer than the plan")
    for s0, s1 in zip(cu, cu[1:]):
        n_tok = s1 - s0
        if n_tok == 0:
            continue
        sl = slice(s0, s1)
        for r0 in range(0, n_tok, plan.chunk_rows):
            n = min(plan.chunk_rows, n_tok - r0)
            indexer_scores(q8[sl], sq[sl], w[sl], k8[sl], sk[sl], r0, n, plan.scores[:n], row_stats=plan.row_stats,
                           stream=stream)
            topk(plan.scores[:n], r0, n, plan.k, plan.idx[r0:r0 + n], max_len=r0 + n, ws=plan.ws,
                 row_stats=plan.row_stats, stream=stream)
        sparse_gqa_prefill(Q[sl], K[sl], V[sl], plan.idx[:n_tok], 0, n_tok, plan.k, sm_scale, O[sl],
                           None if lse is None else lse[sl], stream=stream)
        if idx_out is not None:
            idx_out[sl].copy_(plan.idx[:n_tok])


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

def decode_workspace_size(B, max_seq_len, Hq, Hkv, D, k) -> int:
    return int(lib().dsa_decode_workspace_size(int(B), int(max_seq_len), int(Hq), int(Hkv), int(D), int(k)))


def decode_attention_workspace_size(B, Hq, Hkv, D, k) -> int:
    return int(lib().dsa_decode_attention_workspace_size(int(B), int(Hq), int(Hkv), int(D), int(k)))


def decode_indexer_scores(q8, q_scale, w, k8_cache, k_scale_cache, block_table, seq_lens, max_seq_len, scores,
                          stream=None):
    _need(q8, torch.uint8, 3, "q8")
    _need(k8_cache, torch.uint8, 3, "k8_cache")
    _need(block_table, torch.int32, 2, "block_table")
    _need(scores, torch.float32, 2, "scores")
    B, HI, dI = q8.shape
    _check(lib().dsa_decode_indexer_scores(_ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8_cache), _ptr(k_scale_cache),
                                           _ptr(block_table), block_table.shape[1], k8_cache.shape[0],
                                           _ptr(seq_lens), int(max_seq_len), B, HI, dI, _ptr(scores),
                                           scores.stride(0), _stream(stream)), "dsa_decode_indexer_scores")


def sparse_gqa_decode_attention(q, k_cache, v_cache, block_table, seq_lens, idx, k, sm_scale, ws, out, lse=None,
                                stream=None):
    _need(q, torch.bfloat16, 3, "q")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    _need(out, torch.bfloat16, 3, "out")
    B, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    _check(lib().dsa_sparse_gqa_decode_attention(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                                 block_table.shape[1], k_cache.shape[0], _ptr(seq_lens), _ptr(idx),
                                                 B, Hq, Hkv, D, int(k), float(sm_scale), _ptr(ws),
                                                 ws.numel() * ws.element_size(), _ptr(out), _ptr(lse),
                                                 _stream(stream)), "dsa_sparse_gqa_decode_attention")


def sparse_gqa_decode(q, q8, q_scale, w, k8_cache, k_scale_cache, k_cache, v_cache, block_table, seq_lens,
                      max_seq_len, k, sm_scale, ws, out, idx_out=None, stream=None):
    """dsa_sparse_gqa_decode: indexer -> top-k -> attention for one new token per sequence."""
    _need(q, torch.bfloat16, 3, "q")
    _need(q8, torch.uint8, 3, "q8")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(block_table, torch.int32, 2, "block_table")
    _need(out, torch.bfloat16, 3, "out")
    B, Hq, D = q.shape
    HI, dI = q8.shape[1], q8.shape[2]
    Hkv = k_cache.shape[2]
    _check(lib().dsa_sparse_gqa_decode(_ptr(q), _ptr(q8), _ptr(q_scale), _ptr(w), _ptr(k8_cache),
                                       _ptr(k_scale_cache), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                       block_table.shape[1], k_cache.shape[0], _ptr(seq_lens), int(max_seq_len), B,
                                       Hq, Hkv, D, HI, dI, int(k), float(sm_scale), _ptr(ws),
                                       ws.numel() * ws.element_size(), _ptr(out), _ptr(idx_out), _stream(stream)),
           "dsa_sparse_gqa_decode")


def decode_attention_fixed_scratch_bytes() -> int:
    return int(lib().dsa_decode_attention_fixed_scratch_bytes())


def sparse_gqa_decode_attention_noalloc(q, k_cache, v_cache, block_table, seq_lens, idx, k, sm_scale, out, lse=None,
                                        stream=None):
    """dsa_sparse_gqa_decode_attention_noalloc: the decode attention with no
    caller workspace (its scratch is a fixed array inside the library).  For
    callers that cannot allocate device memory; calls that overlap on one
    GPU race on that array."""
    _need(q, torch.bfloat16, 3, "q")
    _need(k_cache, torch.bfloat16, 4, "k_cache")
    _need(v_cache, torch.bfloat16, 4, "v_cache")
    _need(out, torch.bfloat16, 3, "out")
    B, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    _check(lib().dsa_sparse_gqa_decode_attention_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                                         block_table.shape[1], k_cache.shape[0], _ptr(seq_lens),
                                                         _ptr(idx), B, Hq, Hkv, D, int(k), float(sm_scale),
                                                         _ptr(out), _ptr(lse), _stream(stream)),
           "dsa_sparse_gqa_decode_attention_noalloc")


# ---------------------------------------------------------------------------
# the 8-bit KV cache
# ---------------------------------------------------------------------------

KV8_EXP_MIN = 87  # the least scale exponent byte: 2^-40

_C = torch._C
_U8, _I32, _BF16, _F32 = torch.uint8, torch.int32, torch.bfloat16, torch.float32


def _shaped(t, dtype, shape, name, device):
    """``t`` is a dense tensor of this type and shape on CUDA device ``device``."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected on cuda:{device}, got {t.device}")
    raise ValueError(f"{name}: must be contiguous")


def _device_of(t, name):
    """The index of a tensor's CUDA device."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name}: must be a CUDA tensor")
    return device


def _call(name, device, stream, args):
    """The entry point, on ``device`` (made current if it is not) and on the
    given stream or that device's current one."""
    if stream is None:
        stream = _C._cuda_getCurrentRawStream(device)  # a tenth of what current_stream() costs
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    fn = getattr(_lib or lib(), name)
    if device == _C._cuda_getDevice():
        code = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, stream)
    if code:
        _check(code, name)


def _kv8_cache(k_cache8, v_cache8, kv_exp):
    """Checks the three buffers of an 8-bit cache; (device, num_pages, Hkv, D, scale_block)."""
    device = _device_of(k_cache8, "k_cache8")
    shape = k_cache8.shape
    if len(shape) != 4 or shape[1] != PAGE_SIZE:
        raise ValueError(f"k_cache8: expected [num_pages, {PAGE_SIZE}, Hkv, D], got {tuple(shape)}")
    P, _, Hkv, D = shape
    _shaped(k_cache8, _U8, shape, "k_cache8", device)
    _shaped(v_cache8, _U8, shape, "v_cache8", device)
    parts = kv_exp.shape[1] if kv_exp.dim() == 4 else 0
    if parts not in (1, 2, 4):
        raise ValueError(f"kv_exp: expected [num_pages, 1, 2 or 4, Hkv, 2], got {tuple(kv_exp.shape)}")
    _shaped(kv_exp, _U8, (P, parts, Hkv, 2), "kv_exp", device)
    return device, P, Hkv, D, PAGE_SIZE // parts


def _token_rows(t, n, Hkv, D, name, device):
    """Checks [n, Hkv, D] bf16 rows that may lie apart; the distance in elements."""
    if t.dtype is not _BF16:
        raise TypeError(f"{name}: expected {_BF16}, got {t.dtype}")
    if t.shape != (n, Hkv, D):
        raise ValueError(f"{name}: expected shape {(n, Hkv, D)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected on cuda:{device}, got {t.device}")
    ld, head, one = t.stride()
    if one != 1 or (Hkv > 1 and head != D):
        raise ValueError(f"{name}: a token's [Hkv, D] values must be contiguous")
    return ld if n > 1 else Hkv * D


def _table(block_table, seq_lens, n, device):
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != n:
        raise ValueError(f"block_table: expected [{n}, max_pages], got shape {tuple(shape)}")
    _shaped(block_table, _I32, shape, "block_table", device)
    _shaped(seq_lens, _I32, (n,), "seq_lens", device)
    return shape[1]


def kv8_append(K, V, k_cache8, v_cache8, kv_exp, block_table, seq_lens, cu_seqlens=None, k8=None, k_scale=None,
               k8_cache=None, k_scale_cache=None, stream=None):
    """dsa_kv8_append: new tokens' K and V [n, Hkv, D] bf16 (rows may be parts
    of wider ones) into the 8-bit cache, as the last tokens of sequences whose
    seq_lens [nseq] count them already.  cu_seqlens int32 [nseq+1] for packed
    new tokens, None for one per sequence.  k8 [n, dI] uint8 and k_scale [n]
    float32, with their caches, add the indexer's keys."""
    device, P, Hkv, D, block = _kv8_cache(k_cache8, v_cache8, kv_exp)
    n, nseq = K.shape[0], seq_lens.shape[0]
    ld_k = _token_rows(K, n, Hkv, D, "K", device)
    ld_v = _token_rows(V, n, Hkv, D, "V", device)
    max_pages = _table(block_table, seq_lens, nseq, device)
    if cu_seqlens is not None:
        _shaped(cu_seqlens, _I32, (nseq + 1,), "cu_seqlens", device)
    elif n != nseq:
        raise ValueError(f"K: expected one token for each of {nseq} sequences, got {n}")
    dI = 0
    if k8 is not None:
        if k_scale is None or k8_cache is None or k_scale_cache is None:
            raise ValueError("k8, k_scale, k8_cache and k_scale_cache go together")
        dI = k8.shape[-1]
        _shaped(k8, _U8, (n, dI), "k8", device)
        _shaped(k_scale, _F32, (n,), "k_scale", device)
        _shaped(k8_cache, _U8, (P, PAGE_SIZE, dI), "k8_cache", device)
        _shaped(k_scale_cache, _F32, (P, PAGE_SIZE), "k_scale_cache", device)
    elif k_scale is not None or k8_cache is not None or k_scale_cache is not None:
        raise ValueError("k8, k_scale, k8_cache and k_scale_cache go together")
    _call("dsa_kv8_append", device, stream,
          (K.data_ptr(), ld_k, V.data_ptr(), ld_v, _ptr(k8), _ptr(k_scale), _ptr(cu_seqlens), nseq, n,
           seq_lens.data_ptr(), block_table.data_ptr(), max_pages, P, Hkv, D, dI, block, k_cache8.data_ptr(),
           v_cache8.data_ptr(), kv_exp.data_ptr(), _ptr(k8_cache), _ptr(k_scale_cache)))


def _kv8_rows(q, idx, k, out, lse, Hkv, D, device):
    """Checks the query-side tensors of an attention call; (rows, Hq)."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != D:
        raise ValueError(f"q: expected [rows, Hq, {D}], got shape {tuple(shape)}")
    n, Hq, _ = shape
    _shaped(q, _BF16, shape, "q", device)
    if idx is not None:
        _shaped(idx, _I32, (n, k), "idx", device)
    _shaped(out, _BF16, shape, "out", device)
    if lse is not None:
        _shaped(lse, _F32, (n, Hq), "lse", device)
    return n, Hq


def sparse_gqa_decode_attention_kv8(q, k_cache8, v_cache8, kv_exp, block_table, seq_lens, idx, k, sm_scale, out,
                                    lse=None, stream=None):
    """dsa_sparse_gqa_decode_attention_kv8: attention of each sequence's newest
    token over its selected rows idx [B, k] of the 8-bit cache."""
    device, P, Hkv, D, block = _kv8_cache(k_cache8, v_cache8, kv_exp)
    B, Hq = _kv8_rows(q, idx, int(k), out, lse, Hkv, D, device)
    max_pages = _table(block_table, seq_lens, B, device)
    _call("dsa_sparse_gqa_decode_attention_kv8", device, stream,
          (q.data_ptr(), k_cache8.data_ptr(), v_cache8.data_ptr(), kv_exp.data_ptr(), block, block_table.data_ptr(),
           max_pages, P, seq_lens.data_ptr(), idx.data_ptr(), B, Hq, Hkv, D, int(k), float(sm_scale), out.data_ptr(),
           _ptr(lse)))


def sparse_gqa_prefill_kv8(Q, k_cache8, v_cache8, kv_exp, block_table, seq_lens, idx, cu_seqlens, row_begin, n_rows,
                           k, sm_scale, O, lse=None, stream=None):
    """dsa_sparse_gqa_prefill_kv8: attention of packed query rows [row_begin,
    row_begin+n_rows), the last tokens of their cached sequences, over their
    selected positions in the 8-bit cache.  Q, O, idx and lse hold these rows."""
    device, P, Hkv, D, block = _kv8_cache(k_cache8, v_cache8, kv_exp)
    n, Hq = _kv8_rows(Q, idx, int(k), O, lse, Hkv, D, device)
    if n != int(n_rows):
        raise ValueError(f"Q: expected {int(n_rows)} rows, got {n}")
    nseq = seq_lens.shape[0]
    max_pages = _table(block_table, seq_lens, nseq, device)
    _shaped(cu_seqlens, _I32, (nseq + 1,), "cu_seqlens", device)
    _call("dsa_sparse_gqa_prefill_kv8", device, stream,
          (Q.data_ptr(), k_cache8.data_ptr(), v_cache8.data_ptr(), kv_exp.data_ptr(), block, block_table.data_ptr(),
           max_pages, P, seq_lens.data_ptr(), idx.data_ptr(), _ptr(cu_seqlens), nseq, int(row_begin), n, Hq, Hkv, D,
           int(k), float(sm_scale), O.data_ptr(), _ptr(lse)))


def decode_kv8_workspace_size(B, max_seq_len, k) -> int:
    return int(lib().dsa_decode_kv8_workspace_size(int(B), int(max_seq_len), int(k)))


def sparse_gqa_decode_kv8(q, q8, q_scale, w, k8_cache, k_scale_cache, k_cache8, v_cache8, kv_exp, block_table,
                          seq_lens, max_seq_len, k, sm_scale, ws, out, idx_out=None, stream=None):
    """dsa_sparse_gqa_decode_kv8: indexer -> top-k -> attention over the 8-bit
    cache, for one new token per sequence.  ``ws`` is a uint8 CUDA tensor of
    decode_kv8_workspace_size(...) bytes or more."""
    device, P, Hkv, D, block = _kv8_cache(k_cache8, v_cache8, kv_exp)
    B, Hq = _kv8_rows(q, idx_out, int(k), out, None, Hkv, D, device)
    max_pages = _table(block_table, seq_lens, B, device)
    if q8.dim() != 3:
        raise ValueError(f"q8: expected 3 dims, got shape {tuple(q8.shape)}")
    HI, dI = q8.shape[1], q8.shape[2]
    _shaped(q8, _U8, (B, HI, dI), "q8", device)
    _shaped(q_scale, _F32, (B,), "q_scale", device)
    _shaped(w, _F32, (B, HI), "w", device)
    _shaped(k8_cache, _U8, (P, PAGE_SIZE, dI), "k8_cache", device)
    _shaped(k_scale_cache, _F32, (P, PAGE_SIZE), "k_scale_cache", device)
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor on cuda:{device}")
    _call("dsa_sparse_gqa_decode_kv8", device, stream,
          (q.data_ptr(), q8.data_ptr(), q_scale.data_ptr(), w.data_ptr(), _ptr(k8_cache), _ptr(k_scale_cache),
           k_cache8.data_ptr(), v_cache8.data_ptr(), kv_exp.data_ptr(), block, block_table.data_ptr(), max_pages, P,
           seq_lens.data_ptr(), int(max_seq_len), B, Hq, Hkv, D, HI, dI, int(k), float(sm_scale), ws.data_ptr(),
           ws.nbytes, out.data_ptr(), _ptr(idx_out)))


# ---------------------------------------------------------------------------
# pages of a cache
# ---------------------------------------------------------------------------

_POINTERS = [_P * n for n in range(9)]
_SIZES = [_SZ * n for n in range(9)]


def _page_bufs(bufs, num_pages, device):
    """Host arrays of the buffers' addresses and page sizes; each buffer is a
    dense tensor [num_pages, ...]."""
    n = len(bufs)
    if n > 8 or num_pages < 1:
        raise ValueError(f"bufs: expected at most 8 buffers of at least one page, got {n} of {num_pages}")
    bases, sizes = [], []
    for t in bufs:
        if t.get_device() != device or t.dim() < 1 or t.shape[0] != num_pages or not t.is_contiguous():
            raise ValueError(f"bufs[{len(bases)}]: expected a contiguous tensor of {num_pages} pages on cuda:{device}, "
                             f"got {tuple(t.shape)} on {t.device}")
        bases.append(t.data_ptr())
        sizes.append(t.nbytes // num_pages)
    return _POINTERS[n](*bases), _SIZES[n](*sizes), n


def _pool(block_table, seq_lens, refcount):
    """Checks a pool's state; (device, n_slots, max_pages, num_pages)."""
    device = _device_of(block_table, "block_table")
    n_slots, num_pages = seq_lens.numel(), refcount.numel()
    max_pages = _table(block_table, seq_lens, n_slots, device)
    _shaped(refcount, _I32, (num_pages,), "refcount", device)
    return device, n_slots, max_pages, num_pages


def _entries(device, first, second, third=None):
    """Checks a call's int32 lists (name, tensor) of one length; the length."""
    n = first[1].numel()
    _shaped(first[1], _I32, (n,), first[0], device)
    _shaped(second[1], _I32, (n,), second[0], device)
    if third is not None:
        _shaped(third[1], _I32, (n,), third[0], device)
    return n


def pages_extend(slots, new_lens, block_table, seq_lens, refcount, status, stream=None):
    """dsa_pages_extend: sequence slots[i] grows to new_lens[i] tokens and gets
    the pages that takes; status[i] = 0, or 1 (no pages left) or 2 (refused)."""
    device, n_slots, max_pages, P = _pool(block_table, seq_lens, refcount)
    n = _entries(device, ("slots", slots), ("new_lens", new_lens), ("status", status))
    _call("dsa_pages_extend", device, stream,
          (slots.data_ptr(), new_lens.data_ptr(), n, block_table.data_ptr(), n_slots, max_pages, seq_lens.data_ptr(),
           refcount.data_ptr(), P, status.data_ptr()))


def pages_fork(bufs, parents, children, block_table, seq_lens, refcount, status, stream=None):
    """dsa_pages_fork: the empty slot children[i] becomes a copy of sequence
    parents[i]: full pages shared, a partly filled last page copied in every
    buffer of ``bufs`` (tensors [num_pages, ...]); status as in pages_extend."""
    device, n_slots, max_pages, P = _pool(block_table, seq_lens, refcount)
    n = _entries(device, ("parents", parents), ("children", children), ("status", status))
    bases, sizes, n_bufs = _page_bufs(bufs, P, device)
    _call("dsa_pages_fork", device, stream,
          (bases, sizes, n_bufs, parents.data_ptr(), children.data_ptr(), n, block_table.data_ptr(), n_slots,
           max_pages, seq_lens.data_ptr(), refcount.data_ptr(), P, status.data_ptr()))


def pages_free(slots, block_table, seq_lens, refcount, stream=None):
    """dsa_pages_free: the sequences in ``slots`` become empty and pages that no
    other sequence holds become free."""
    device, n_slots, max_pages, P = _pool(block_table, seq_lens, refcount)
    n = slots.numel()
    _shaped(slots, _I32, (n,), "slots", device)
    _call("dsa_pages_free", device, stream,
          (slots.data_ptr(), n, block_table.data_ptr(), n_slots, max_pages, seq_lens.data_ptr(), refcount.data_ptr(),
           P))


def pages_copy(bufs, src, dst, stream=None):
    """dsa_pages_copy: page src[i] to page dst[i] in every buffer of ``bufs``
    (tensors [num_pages, ...])."""
    if not bufs:
        raise ValueError("bufs: expected at least one buffer")
    device = _device_of(bufs[0], "bufs[0]")
    if bufs[0].dim() < 1:
        raise ValueError("bufs[0]: expected [num_pages, ...]")
    P = bufs[0].shape[0]
    n = _entries(device, ("src", src), ("dst", dst))
    bases, sizes, n_bufs = _page_bufs(bufs, P, device)
    _call("dsa_pages_copy", device, stream,
          (bases, sizes, n_bufs, src.data_ptr(), dst.data_ptr(), n, P))


def pages_compact_workspace_size(num_pages) -> int:
    return int(lib().dsa_pages_compact_workspace_size(int(num_pages)))


def pages_compact(bufs, block_table, seq_lens, refcount, page_map, n_used, ws, block_table_out=None,
                  refcount_out=None, stream=None):
    """dsa_pages_compact: the pages in use come to the lowest ids, in every
    buffer of ``bufs``; page_map [num_pages] int32 receives the new ids (-1:
    free), n_used [1] int32 their number.  The table and the counts change in
    place unless other tensors are given for them."""
    device, n_slots, max_pages, P = _pool(block_table, seq_lens, refcount)
    table_out = block_table if block_table_out is None else block_table_out
    refs_out = refcount if refcount_out is None else refcount_out
    _shaped(table_out, _I32, (n_slots, max_pages), "block_table_out", device)
    _shaped(refs_out, _I32, (P,), "refcount_out", device)
    _shaped(page_map, _I32, (P,), "page_map", device)
    _shaped(n_used, _I32, (1,), "n_used", device)
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor on cuda:{device}")
    bases, sizes, n_bufs = _page_bufs(bufs, P, device)
    _call("dsa_pages_compact", device, stream,
          (bases, sizes, n_bufs, block_table.data_ptr(), table_out.data_ptr(), n_slots, max_pages,
           seq_lens.data_ptr(), refcount.data_ptr(), refs_out.data_ptr(), P, page_map.data_ptr(), n_used.data_ptr(),
           ws.data_ptr(), ws.nbytes))


class KV8Cache:
    """Buffers of an 8-bit paged cache and of its pool of pages: K and V
    (``k``, ``v``, ``exp``), the indexer's keys (``k8``, ``k_scale``; with dI),
    and the pool's ``block_table``, ``seq_lens`` and ``refcount``.

    The methods call the functions of this module on the current stream.
    ``slots`` is an int32 CUDA tensor of the sequences that take part, in the
    order of the batch (one out of range takes part as an empty sequence); None
    means every slot in order."""

    def __init__(self, num_pages, n_slots, max_pages, Hkv, D, dI=None, scale_block=64, device="cuda"):
        if scale_block not in (16, 32, 64):
            raise ValueError(f"scale_block: expected 16, 32 or 64, got {scale_block}")
        e8 = dict(dtype=torch.uint8, device=device)
        e32 = dict(dtype=torch.int32, device=device)
        self.k = torch.zeros(num_pages, PAGE_SIZE, Hkv, D, **e8)
        self.v = torch.zeros(num_pages, PAGE_SIZE, Hkv, D, **e8)
        self.exp = torch.full((num_pages, PAGE_SIZE // scale_block, Hkv, 2), KV8_EXP_MIN, **e8)
        self.k8 = torch.zeros(num_pages, PAGE_SIZE, dI, **e8) if dI else None
        self.k_scale = torch.ones(num_pages, PAGE_SIZE, dtype=torch.float32, device=device) if dI else None
        self.block_table = torch.full((n_slots, max_pages), -1, **e32)
        self.seq_lens = torch.zeros(n_slots, **e32)
        self.refcount = torch.zeros(num_pages, **e32)
        self.bufs = [t for t in (self.k, self.v, self.exp, self.k8, self.k_scale) if t is not None]

    def _rows(self, slots):
        if slots is None:
            return self.block_table, self.seq_lens
        rows = slots.clamp(0, self.seq_lens.numel() - 1)
        lens = self.seq_lens.index_select(0, rows)
        return self.block_table.index_select(0, rows), torch.where(rows == slots, lens, torch.zeros_like(lens))

    def extend(self, slots, new_lens):
        """pages_extend; the status tensor."""
        status = torch.empty_like(slots)
        pages_extend(slots, new_lens, self.block_table, self.seq_lens, self.refcount, status)
        return status

    def fork(self, parents, children):
        """pages_fork; the status tensor."""
        status = torch.empty_like(children)
        pages_fork(self.bufs, parents, children, self.block_table, self.seq_lens, self.refcount, status)
        return status

    def free(self, slots):
        pages_free(slots, self.block_table, self.seq_lens, self.refcount)

    def compact(self):
        """pages_compact in place; (page_map, n_used)."""
        page_map = torch.empty_like(self.refcount)
        n_used = torch.empty(1, dtype=torch.int32, device=self.refcount.device)
        ws = torch.empty(pages_compact_workspace_size(len(self.refcount)), dtype=torch.uint8,
                         device=self.refcount.device)
        pages_compact(self.bufs, self.block_table, self.seq_lens, self.refcount, page_map, n_used, ws)
        return page_map, n_used

    def append(self, K, V, cu_seqlens=None, k8=None, k_scale=None, slots=None):
        """kv8_append of the last tokens of the sequences (extend comes first).
        k8 and k_scale are given exactly when the cache holds indexer keys: a
        page's earlier keys are another sequence's.  A slot is named once."""
        if (self.k8 is None) != (k8 is None):
            raise ValueError("k8: the cache holds " + ("no indexer keys (dI)" if self.k8 is None else
                                                       "indexer keys (dI), and these tokens come without"))
        table, lens = self._rows(slots)
        kv8_append(K, V, self.k, self.v, self.exp, table, lens, cu_seqlens, k8, k_scale, self.k8, self.k_scale)

    def prefill(self, Q, idx, cu_seqlens, O, sm_scale=None, lse=None, slots=None):
        """sparse_gqa_prefill_kv8 of all packed query rows."""
        table, lens = self._rows(slots)
        scale = 1.0 / math.sqrt(Q.shape[2]) if sm_scale is None else sm_scale
        sparse_gqa_prefill_kv8(Q, self.k, self.v, self.exp, table, lens, idx, cu_seqlens, 0, Q.shape[0],
                               idx.shape[1], scale, O, lse)

    def decode(self, q, q8, q_scale, w, max_seq_len, k, ws, out, sm_scale=None, idx_out=None, slots=None):
        """sparse_gqa_decode_kv8 of one new token per sequence."""
        if self.k8 is None:
            raise ValueError("the cache holds no indexer keys (dI)")
        table, lens = self._rows(slots)
        scale = 1.0 / math.sqrt(q.shape[2]) if sm_scale is None else sm_scale
        sparse_gqa_decode_kv8(q, q8, q_scale, w, self.k8, self.k_scale, self.k, self.v, self.exp, table, lens,
                              max_seq_len, k, scale, ws, out, idx_out)


# ---------------------------------------------------------------------------
# diagnostics
# ---------------------------------------------------------------------------

def read_probe(buf, reps, sink, stream=None):
    """dsa_read_probe: read ``buf`` (a contiguous CUDA tensor, 16-byte
    multiple) ``reps`` times with L2-only 16-byte loads.  For timing the
    memory system's read bandwidth; ``sink`` is a small CUDA tensor the kernel
    may write."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous CUDA tensor")
    _check(lib().dsa_read_probe(_ptr(buf), buf.numel() * buf.element_size(), int(reps), _ptr(sink),
                                _stream(stream)), "dsa_read_probe")
