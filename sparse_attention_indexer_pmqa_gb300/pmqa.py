"""ctypes binding of libpmqa (include/pmqa.h). Argument marshalling only.

Functions carry the C names. Tensors are torch CUDA tensors; torch supplies
device memory and the current stream, every step of the computation runs in
the library's kernels. There is no CPU path: if the library is missing,
``load()`` raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

from . import build as _build

PMQA_OK = 0
PMQA_ERR_INVALID_ARG = -1
PMQA_ERR_UNSUPPORTED = -2
PMQA_ERR_WORKSPACE = -3
PMQA_ERR_CUDA = -4
PMQA_ERR_DEVICE = -5

PMQA_DEV_BAD_BLOCK_ID = 0x1
PMQA_DEV_BAD_CONTEXT = 0x2
PMQA_DEV_TIMEOUT = 0x4
PMQA_DEV_OVERFLOW = 0x8
PMQA_DEV_INTERNAL = 0x10
PMQA_DEV_SCORE_RANGE = 0x20

PMQA_OP_LOGITS = 0
PMQA_OP_TOPK = 1
PMQA_OP_LOGITS_TOPK = 2
PMQA_OP_MQA_LOGITS = 3

PMQA_ROPE_PLAIN = 0
PMQA_ROPE_LINEAR = 1
PMQA_ROPE_PARTS = 2

PMQA_NORM_NONE = 0
PMQA_NORM_LAYER = 1
PMQA_NORM_RMS = 2

PMQA_STAGE_SCORE = 1
PMQA_STAGE_SELECT = 2

EXPORTED = (
    "pmqa_workspace_bytes", "pmqa_workspace_init", "pmqa_logits", "pmqa_topk",
    "pmqa_logits_topk", "pmqa_logits_topk_stages", "pmqa_logits_topk_noalloc",
    "pmqa_logits_topk_range",
    "pmqa_mqa_logits", "pmqa_topk_merge", "pmqa_sparse_mla_workspace_bytes",
    "pmqa_sparse_mla_decode", "pmqa_sparse_mla_decode_range", "pmqa_sparse_mla_merge",
    "pmqa_cache_workspace_bytes", "pmqa_cache_append", "pmqa_cache_attention",
    "pmqa_cache_weigh", "pmqa_cache_evict",
    "pmqa_rope_frequencies", "pmqa_rope", "pmqa_index_append", "pmqa_index_read",
    "pmqa_latent_append", "pmqa_latent_workspace_bytes", "pmqa_latent_attention",
    "pmqa_gather_probe", "pmqa_read_device_status", "pmqa_status_string", "pmqa_version",
)


class PmqaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {code} ({status_string(code)})")


class Problem(ctypes.Structure):
    """Mirror of struct pmqa_problem."""

    _fields_ = [
        ("q", ctypes.c_void_p),
        ("kv_cache", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("context_lens", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p),
        ("bs", ctypes.c_int32),
        ("next_n", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("max_model_len", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64),
    ]


class MqaProblem(ctypes.Structure):
    """Mirror of struct pmqa_mqa_problem."""

    _fields_ = [
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("ks", ctypes.c_void_p),
        ("ke", ctypes.c_void_p),
        ("m", ctypes.c_int32),
        ("n", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
    ]


class MlaProblem(ctypes.Structure):
    """Mirror of struct pmqa_mla_problem."""

    _fields_ = [
        ("q", ctypes.c_void_p),
        ("kv_cache", ctypes.c_void_p),
        ("indices", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p),
        ("q_scale", ctypes.c_float),
        ("kv_scale", ctypes.c_float),
        ("sm_scale", ctypes.c_float),
        ("bs", ctypes.c_int32),
        ("next_n", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("v_head_dim", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64),
    ]


class CacheProblem(ctypes.Structure):
    """Mirror of struct pmqa_cache_problem."""

    _fields_ = [
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p),
        ("context_lens", ctypes.c_void_p),
        ("row_begin", ctypes.c_void_p),
        ("bs", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("rows", ctypes.c_int32),
        ("max_rows", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64),
    ]


class PagedRows(ctypes.Structure):
    """Mirror of struct pmqa_paged_rows."""

    _fields_ = [
        ("block_tables", ctypes.c_void_p),
        ("context_lens", ctypes.c_void_p),
        ("row_begin", ctypes.c_void_p),
        ("bs", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("rows", ctypes.c_int32),
        ("max_rows", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64),
    ]


class RotaryArgs(ctypes.Structure):
    """Mirror of struct pmqa_rotary."""

    _fields_ = [
        ("inv_freq", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("dim", ctypes.c_int32),
        ("begin", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class Heads(ctypes.Structure):
    """Mirror of struct pmqa_heads."""

    _fields_ = [
        ("x", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("x_row", ctypes.c_int64),
        ("x_head", ctypes.c_int64),
        ("out_row", ctypes.c_int64),
        ("out_head", ctypes.c_int64),
        ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
    ]


class NormArgs(ctypes.Structure):
    """Mirror of struct pmqa_norm."""

    _fields_ = [
        ("kind", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("weight", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
    ]


class IndexRows(ctypes.Structure):
    """Mirror of struct pmqa_index_rows."""

    _fields_ = [
        ("k", ctypes.c_void_p),
        ("q", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p),
        ("weights_out", ctypes.c_void_p),
        ("k_row", ctypes.c_int64),
        ("q_row", ctypes.c_int64),
        ("q_head", ctypes.c_int64),
        ("weights_row", ctypes.c_int64),
        ("heads", ctypes.c_int32),
        ("weights_bf16", ctypes.c_int32),
        ("weight_scale", ctypes.c_float),
    ]


class LatentRows(ctypes.Structure):
    """Mirror of struct pmqa_latent_rows."""

    _fields_ = [
        ("c", ctypes.c_void_p),
        ("k_pe", ctypes.c_void_p),
        ("q_c", ctypes.c_void_p),
        ("q_pe", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p),
        ("c_row", ctypes.c_int64),
        ("pe_row", ctypes.c_int64),
        ("q_c_row", ctypes.c_int64),
        ("q_c_head", ctypes.c_int64),
        ("q_pe_row", ctypes.c_int64),
        ("q_pe_head", ctypes.c_int64),
        ("heads", ctypes.c_int32),
        ("kv_scale", ctypes.c_float),
        ("q_scale", ctypes.c_float),
    ]


class Rotary(NamedTuple):
    """Rotary positions of the values begin .. begin + dim of a head: inv_freq is a
    float64 tensor [dim / 2] on the device (see rope_frequencies)."""

    inv_freq: object
    begin: int = 0
    interleaved: bool = False
    scale: float = 1.0


class Norm(NamedTuple):
    """Normalisation of a row: kind PMQA_NORM_*, weight and bias float32 tensors of
    the row's width or None."""

    kind: int
    weight: object = None
    bias: object = None
    eps: float = 1e-6


_lib = None
_torch_names = ()


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libpmqa.so (built by build.build()); raise if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise FileNotFoundError(
            f"{path} is missing: build it with sparse_attention_indexer_pmqa_gb300.build.build()")
    lib = ctypes.CDLL(path)
    V, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    PP = ctypes.POINTER(Problem)
    PM = ctypes.POINTER(MqaProblem)
    PL = ctypes.POINTER(MlaProblem)
    PC = ctypes.POINTER(CacheProblem)
    PR, PO = ctypes.POINTER(PagedRows), ctypes.POINTER(RotaryArgs)
    PH, PN = ctypes.POINTER(Heads), ctypes.POINTER(NormArgs)
    F32, F64 = ctypes.c_float, ctypes.c_double
    sig = {
        "pmqa_workspace_bytes": ([I32, I32, I32, I32, ctypes.c_int], SZ),
        "pmqa_workspace_init": ([V, SZ, V], ctypes.c_int),
        "pmqa_logits": ([PP, V, V, SZ, V], ctypes.c_int),
        "pmqa_topk": ([V, V, I32, I32, I32, I32, V, V, V, SZ, V], ctypes.c_int),
        "pmqa_logits_topk": ([PP, I32, V, V, V, V, SZ, V], ctypes.c_int),
        "pmqa_logits_topk_stages": ([PP, I32, V, V, V, V, SZ, V, I32], ctypes.c_int),
        "pmqa_logits_topk_noalloc": ([PP, I32, V, V, V, V], ctypes.c_int),
        "pmqa_logits_topk_range": ([PP, V, V, I32, V, V, V, SZ, V], ctypes.c_int),
        "pmqa_mqa_logits": ([PM, V, V, SZ, V], ctypes.c_int),
        "pmqa_topk_merge": ([V, V, I32, I32, I32, I32, V, V, V], ctypes.c_int),
        "pmqa_sparse_mla_workspace_bytes": ([I32], SZ),
        "pmqa_sparse_mla_decode": ([PL, V, V, V, SZ, V], ctypes.c_int),
        "pmqa_sparse_mla_decode_range": ([PL, V, V, V, V, V, SZ, V], ctypes.c_int),
        "pmqa_sparse_mla_merge": ([V, V, I32, I32, I32, V, V, V], ctypes.c_int),
        "pmqa_cache_workspace_bytes": ([], SZ),
        "pmqa_cache_append": ([PC, V, V, V, SZ, V], ctypes.c_int),
        "pmqa_cache_attention": ([PC, V, I32, F32, V, V, V, SZ, V], ctypes.c_int),
        "pmqa_cache_weigh": ([PC, V, I32, F32, V, V, V, I64, V, SZ, V], ctypes.c_int),
        "pmqa_cache_evict": ([PC, V, I64, I32, I32, I32, V, I32, V, V, V, V, SZ, V],
                             ctypes.c_int),
        "pmqa_rope_frequencies": ([I32, F64, ctypes.c_int, F64, F64, F64, F64,
                                   ctypes.POINTER(F64), ctypes.POINTER(F32)], ctypes.c_int),
        "pmqa_rope": ([PO, I32, PH, PH, V], ctypes.c_int),
        "pmqa_index_append": ([PR, V, ctypes.POINTER(IndexRows), PN, PO, V, SZ, V], ctypes.c_int),
        "pmqa_index_read": ([PR, V, V, V, V, V, SZ, V], ctypes.c_int),
        "pmqa_latent_append": ([PR, V, ctypes.POINTER(LatentRows), PN, PO, V, SZ, V],
                               ctypes.c_int),
        "pmqa_latent_workspace_bytes": ([], SZ),
        "pmqa_latent_attention": ([PR, V, V, I32, F32, F32, F32, V, V, V, SZ, V], ctypes.c_int),
        "pmqa_gather_probe": ([V, ctypes.c_uint64, V, I64, I32, I32, V, V], ctypes.c_int),
        "pmqa_read_device_status": ([V, V], ctypes.c_int),
        "pmqa_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "pmqa_version": ([], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().pmqa_status_string(code).decode()


def _stream(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(code: int, what: str) -> None:
    if code != PMQA_OK:
        raise PmqaError(code, what)


def make_problem(q, kv_cache, weights, context_lens, block_tables, max_model_len: int) -> Problem:
    """Fill a pmqa_problem from tensors shaped as in the C header."""
    bs, next_n, heads, head_dim = q.shape
    num_blocks, block_size = kv_cache.shape[0], kv_cache.shape[1]
    assert kv_cache.shape[-1] == head_dim + 4, "kv rows hold head_dim fp8 bytes + fp32 scale"
    for t in (q, kv_cache, weights, context_lens, block_tables):
        assert t.is_cuda and t.is_contiguous()
    return Problem(
        q=q.data_ptr(), kv_cache=kv_cache.data_ptr(), weights=weights.data_ptr(),
        context_lens=context_lens.data_ptr(), block_tables=block_tables.data_ptr(),
        bs=bs, next_n=next_n, heads=heads, head_dim=head_dim, block_size=block_size,
        max_blocks_per_seq=block_tables.shape[1], max_model_len=max_model_len,
        num_blocks=num_blocks)


def pmqa_workspace_bytes(bs: int, next_n: int, max_model_len: int, k: int, op: int) -> int:
    return int(load().pmqa_workspace_bytes(bs, next_n, max_model_len, k, op))


def workspace(bs: int, next_n: int, max_model_len: int, k: int, op: int, device=None, stream=None):
    """A zero-initialised workspace tensor for the given operation."""
    import torch

    n = pmqa_workspace_bytes(bs, next_n, max_model_len, k, op)
    if n == 0:
        raise PmqaError(PMQA_ERR_INVALID_ARG, "pmqa_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    pmqa_workspace_init(ws, stream=stream)
    return ws


def pmqa_workspace_init(ws, stream=None) -> None:
    _check(load().pmqa_workspace_init(_ptr(ws), ws.numel(), _stream(stream)),
           "pmqa_workspace_init")


def pmqa_logits(q, kv_cache, weights, context_lens, block_tables, max_model_len: int, *,
                out=None, ws=None, stream=None):
    """fp32 logits [bs*next_n, max_model_len]."""
    import torch

    p = make_problem(q, kv_cache, weights, context_lens, block_tables, max_model_len)
    rows = p.bs * p.next_n
    if out is None:
        out = torch.empty((rows, max_model_len), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(p.bs, p.next_n, max_model_len, 0, PMQA_OP_LOGITS, q.device, stream)
    _check(load().pmqa_logits(ctypes.byref(p), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "pmqa_logits")
    return out


def pmqa_topk(logits, context_lens, next_n: int, k: int, *, idx=None, vals=None,
              want_vals: bool = False, ws=None, stream=None):
    """int32 positions [rows, k] (and fp32 values) of each row's top-k."""
    import torch

    rows, mml = logits.shape
    bs = context_lens.shape[0]
    assert rows == bs * next_n
    if idx is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=logits.device)
    if vals is None and want_vals:
        vals = torch.empty((rows, k), dtype=torch.float32, device=logits.device)
    if ws is None:
        ws = workspace(bs, next_n, mml, k, PMQA_OP_TOPK, logits.device, stream)
    _check(load().pmqa_topk(_ptr(logits), _ptr(context_lens), bs, next_n, mml, k, _ptr(idx),
                            _ptr(vals), _ptr(ws), ws.numel(), _stream(stream)), "pmqa_topk")
    return (idx, vals) if want_vals or vals is not None else idx


def pmqa_logits_topk(q, kv_cache, weights, context_lens, block_tables, max_model_len: int,
                     k: int, *, idx=None, vals=None, logits=None, want_vals: bool = False,
                     ws=None, stream=None):
    """Fused logits + top-k; returns idx, or (idx, vals) when values are asked for."""
    import torch

    p = make_problem(q, kv_cache, weights, context_lens, block_tables, max_model_len)
    rows = p.bs * p.next_n
    if idx is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((rows, k), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(p.bs, p.next_n, max_model_len, k, PMQA_OP_LOGITS_TOPK, q.device, stream)
    _check(load().pmqa_logits_topk(ctypes.byref(p), k, _ptr(idx), _ptr(vals), _ptr(logits),
                                   _ptr(ws), ws.numel(), _stream(stream)), "pmqa_logits_topk")
    return (idx, vals) if want_vals or vals is not None else idx


def pmqa_logits_topk_stages(q, kv_cache, weights, context_lens, block_tables, max_model_len: int,
                            k: int, stages: int, *, idx, ws, vals=None, logits=None,
                            stream=None):
    """One or both launches of the fused call (PMQA_STAGE_SCORE, then
    PMQA_STAGE_SELECT with the same arguments and workspace)."""
    p = make_problem(q, kv_cache, weights, context_lens, block_tables, max_model_len)
    _check(load().pmqa_logits_topk_stages(ctypes.byref(p), k, _ptr(idx), _ptr(vals), _ptr(logits),
                                          _ptr(ws), ws.numel(), _stream(stream), stages),
           "pmqa_logits_topk_stages")
    return idx


def pmqa_logits_topk_noalloc(q, kv_cache, weights, context_lens, block_tables,
                             max_model_len: int, k: int, *, idx, vals=None, logits=None,
                             stream=None):
    """Fused logits + top-k with the library's built-in device scratch; the
    caller passes every output buffer, nothing is allocated."""
    p = make_problem(q, kv_cache, weights, context_lens, block_tables, max_model_len)
    _check(load().pmqa_logits_topk_noalloc(ctypes.byref(p), k, _ptr(idx), _ptr(vals), _ptr(logits),
                                           _stream(stream)), "pmqa_logits_topk_noalloc")
    return idx


def pmqa_logits_topk_range(q, kv_cache, weights, context_lens, block_tables, max_model_len: int,
                           k: int, token_begin, token_end, *, idx=None, vals=None,
                           want_vals: bool = False, ws=None, stream=None):
    """The fused call on the slice [token_begin[i], token_end[i]) of each
    request's tokens; positions in idx are the requests' own (global) ones."""
    import torch

    p = make_problem(q, kv_cache, weights, context_lens, block_tables, max_model_len)
    rows = p.bs * p.next_n
    for t in (token_begin, token_end):
        assert t.is_cuda and t.is_contiguous() and t.dtype == torch.int32 and t.numel() == p.bs
    if idx is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((rows, k), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(p.bs, p.next_n, max_model_len, k, PMQA_OP_LOGITS_TOPK, q.device, stream)
    _check(load().pmqa_logits_topk_range(ctypes.byref(p), _ptr(token_begin), _ptr(token_end), k,
                                         _ptr(idx), _ptr(vals), _ptr(ws), ws.numel(),
                                         _stream(stream)), "pmqa_logits_topk_range")
    return (idx, vals) if want_vals or vals is not None else idx


def make_mqa_problem(q, k, k_scale, weights, ks, ke) -> MqaProblem:
    """Fill a pmqa_mqa_problem from tensors shaped as in the C header."""
    m, heads, head_dim = q.shape
    n = k.shape[0]
    assert k.shape[1] == head_dim and k_scale.shape[0] == n
    for t in (q, k, k_scale, weights, ks, ke):
        assert t.is_cuda and t.is_contiguous()
    return MqaProblem(q=q.data_ptr(), k=k.data_ptr(), k_scale=k_scale.data_ptr(),
                      weights=weights.data_ptr(), ks=ks.data_ptr(), ke=ke.data_ptr(),
                      m=m, n=n, heads=heads, head_dim=head_dim)


def pmqa_mqa_logits(q, k, k_scale, weights, ks, ke, *, out=None, ws=None, stream=None):
    """Prefill logits fp32 [m, n] over the rows' key ranges [ks, ke)."""
    import torch

    p = make_mqa_problem(q, k, k_scale, weights, ks, ke)
    if out is None:
        out = torch.empty((p.m, p.n), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(p.m, 1, p.n, 0, PMQA_OP_MQA_LOGITS, q.device, stream)
    _check(load().pmqa_mqa_logits(ctypes.byref(p), _ptr(out), _ptr(ws), ws.numel(),
                                  _stream(stream)), "pmqa_mqa_logits")
    return out


def pmqa_topk_merge(idx, vals, k: int, *, out_idx=None, out_vals=None, want_vals: bool = False,
                    stream=None):
    """Top-k per row of the union of candidate lists idx/vals [lists, rows, k_in]
    (-1 marks an empty slot); returns out_idx [rows, k] (and out_vals)."""
    import torch

    lists, rows, k_in = idx.shape
    assert vals.shape == idx.shape and idx.is_contiguous() and vals.is_contiguous()
    if out_idx is None:
        out_idx = torch.empty((rows, k), dtype=torch.int32, device=idx.device)
    if out_vals is None and want_vals:
        out_vals = torch.empty((rows, k), dtype=torch.float32, device=idx.device)
    _check(load().pmqa_topk_merge(_ptr(idx), _ptr(vals), lists, rows, k_in, k, _ptr(out_idx),
                                  _ptr(out_vals), _stream(stream)), "pmqa_topk_merge")
    return (out_idx, out_vals) if want_vals or out_vals is not None else out_idx


def make_mla_problem(q, kv_cache, indices, block_tables, next_n: int, q_scale: float,
                     kv_scale: float, sm_scale: float) -> MlaProblem:
    """Fill a pmqa_mla_problem from tensors shaped as in the C header (q may
    also be given as [bs, next_n, heads, 576])."""
    bs = block_tables.shape[0]
    heads, head_dim = q.shape[-2], q.shape[-1]
    rows = q.numel() // (heads * head_dim)
    assert rows == bs * next_n and indices.shape[0] == rows
    num_blocks, block_size = kv_cache.shape[0], kv_cache.shape[1]
    assert kv_cache.shape[-1] == head_dim
    for t in (q, kv_cache, indices, block_tables):
        assert t.is_cuda and t.is_contiguous()
    return MlaProblem(q=q.data_ptr(), kv_cache=kv_cache.data_ptr(), indices=indices.data_ptr(),
                      block_tables=block_tables.data_ptr(), q_scale=q_scale, kv_scale=kv_scale,
                      sm_scale=sm_scale, bs=bs, next_n=next_n, heads=heads, head_dim=head_dim,
                      v_head_dim=512, topk=indices.shape[1], block_size=block_size,
                      max_blocks_per_seq=block_tables.shape[1], num_blocks=num_blocks)


def pmqa_sparse_mla_workspace_bytes(rows: int) -> int:
    return int(load().pmqa_sparse_mla_workspace_bytes(rows))


def mla_workspace(rows: int, device=None, stream=None):
    """A zero-initialised workspace for pmqa_sparse_mla_decode."""
    import torch

    n = pmqa_sparse_mla_workspace_bytes(rows)
    if n == 0:
        raise PmqaError(PMQA_ERR_INVALID_ARG, "pmqa_sparse_mla_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    pmqa_workspace_init(ws, stream=stream)
    return ws


def pmqa_sparse_mla_decode(q, kv_cache, indices, block_tables, next_n: int, q_scale: float,
                           kv_scale: float, sm_scale: float, *, out=None, lse=None,
                           want_lse: bool = False, ws=None, stream=None):
    """Sparse MLA decode over the listed positions: bf16 out [rows, heads, 512]
    (and fp32 lse [rows, heads] when asked for or given)."""
    import torch

    p = make_mla_problem(q, kv_cache, indices, block_tables, next_n, q_scale, kv_scale, sm_scale)
    rows = p.bs * p.next_n
    if out is None:
        out = torch.empty((rows, p.heads, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((rows, p.heads), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = mla_workspace(rows, q.device, stream)
    _check(load().pmqa_sparse_mla_decode(ctypes.byref(p), _ptr(out), _ptr(lse), _ptr(ws),
                                         ws.numel(), _stream(stream)), "pmqa_sparse_mla_decode")
    return (out, lse) if want_lse or lse is not None else out


def pmqa_sparse_mla_decode_range(q, kv_cache, indices, block_tables, next_n: int, q_scale: float,
                                 kv_scale: float, sm_scale: float, token_begin, token_end, *,
                                 out=None, lse=None, ws=None, stream=None):
    """The decode over each request's slice [token_begin[i], token_end[i]) of
    its tokens: (bf16 out [rows, heads, 512], fp32 lse [rows, heads])."""
    import torch

    p = make_mla_problem(q, kv_cache, indices, block_tables, next_n, q_scale, kv_scale, sm_scale)
    rows = p.bs * p.next_n
    for t in (token_begin, token_end):
        assert t.is_cuda and t.is_contiguous() and t.dtype == torch.int32 and t.numel() == p.bs
    if out is None:
        out = torch.empty((rows, p.heads, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((rows, p.heads), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = mla_workspace(rows, q.device, stream)
    _check(load().pmqa_sparse_mla_decode_range(ctypes.byref(p), _ptr(token_begin), _ptr(token_end),
                                               _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                               _stream(stream)), "pmqa_sparse_mla_decode_range")
    return out, lse


def pmqa_sparse_mla_merge(outs, lses, *, out=None, lse=None, stream=None):
    """LSE-weighted merge of partial decodes outs [parts, rows, heads, 512]
    (bf16) with lses [parts, rows, heads]; returns (out, lse)."""
    import torch

    parts, rows, heads, vdim = outs.shape
    assert lses.shape == (parts, rows, heads) and vdim == 512
    assert outs.is_contiguous() and lses.is_contiguous() and outs.dtype == torch.bfloat16
    if out is None:
        out = torch.empty((rows, heads, vdim), dtype=torch.bfloat16, device=outs.device)
    if lse is None:
        lse = torch.empty((rows, heads), dtype=torch.float32, device=outs.device)
    _check(load().pmqa_sparse_mla_merge(_ptr(outs), _ptr(lses), parts, rows, heads, _ptr(out),
                                        _ptr(lse), _stream(stream)), "pmqa_sparse_mla_merge")
    return out, lse


def make_cache_problem(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                       row_begin=None, rows: int = 0, max_rows: int = 0) -> CacheProblem:
    """Fill a pmqa_cache_problem from tensors shaped as in the C header (the
    pools as float8_e4m3fn or uint8; v_cache and v_scale may be None where the
    call does not read values)."""
    num_blocks, kv_heads, block_size, head_dim = pool = k_cache.shape
    bs, width = block_tables.shape
    dev = k_cache.get_device()
    f32, i32, _, _, _, codes, _, _ = _torch()
    code = k_cache.dtype
    if code not in codes or not k_cache.is_contiguous():
        raise AssertionError(f"expected contiguous float8_e4m3fn (or uint8) pools, got {code}")
    _like(k_scale, dev, f32, (num_blocks, kv_heads))
    if v_cache is not None:
        _like(v_cache, dev, code, pool)
        _like(v_scale, dev, f32, (num_blocks, kv_heads))
    _like(block_tables, dev, i32, (bs, width))
    _like(context_lens, dev, i32, (bs,))
    if row_begin is not None:
        _like(row_begin, dev, i32, (bs + 1,))
    return CacheProblem(
        k_cache.data_ptr(), None if v_cache is None else v_cache.data_ptr(), k_scale.data_ptr(),
        None if v_cache is None else v_scale.data_ptr(), block_tables.data_ptr(),
        context_lens.data_ptr(), None if row_begin is None else row_begin.data_ptr(),
        bs, kv_heads, head_dim, block_size, width, rows, max_rows, num_blocks)


def pmqa_cache_workspace_bytes() -> int:
    return int(load().pmqa_cache_workspace_bytes())


def cache_workspace(device=None, stream=None):
    """A zero-initialised workspace for the pmqa_cache_* calls. With a `stream` the
    memory is that stream's too: it may be in use on the current one."""
    import torch

    with torch.cuda.stream(stream):
        ws = torch.empty(pmqa_cache_workspace_bytes(), dtype=torch.uint8, device=device or "cuda")
        with torch.cuda.device(ws.device):
            pmqa_workspace_init(ws, stream=stream)
    return ws


def _torch():
    """torch's float32, int32 and bfloat16, the calls that name the current device
    and its stream's handle, the pools' types, float64 and torch.empty (torch is
    imported on first use)."""
    global _torch_names
    if not _torch_names:
        import torch

        _torch_names = (torch.float32, torch.int32, torch.bfloat16, torch._C._cuda_getDevice,
                        torch._C._cuda_getCurrentRawStream,
                        (torch.float8_e4m3fn, torch.uint8), torch.float64, torch.empty)
    return _torch_names


def _like(t, dev: int, dtype, shape) -> None:
    """What every operand of a call on a cache must be: on the cache's
    device, of the documented type and shape, contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise AssertionError(f"expected a contiguous {dtype} tensor of shape {tuple(shape)} on the "
                             f"cache's device ({dev}), got {tuple(t.shape)} {t.dtype} on {t.device}")


def _on_stream(fn):
    """With a `stream`, everything that the call allocates, fills or copies is
    that stream's too."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch

        with torch.cuda.stream(stream):
            return fn(*args, stream=stream, **kw)
    return call


def _cache_call(name: str, p: CacheProblem, dev: int, stream, ws, *args) -> None:
    """Call a pmqa_cache_* function with device `dev` current, on its current
    stream unless one is given."""
    if dev < 0:
        raise AssertionError("the pmqa_cache_* calls take cuda tensors")
    current_device, raw_stream = _torch()[3:5]
    if dev != current_device():
        import torch

        with torch.cuda.device(dev):
            return _cache_call(name, p, dev, stream, ws, *args)
    if ws is None:
        ws = cache_workspace(f"cuda:{dev}", stream)
    if ws.get_device() != dev or not ws.is_contiguous():
        raise AssertionError("expected a contiguous workspace on the cache's device")
    rc = getattr(_lib or load(), name)(p, *args, ws.data_ptr(), ws.nbytes,
                                       raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc != PMQA_OK:
        raise PmqaError(rc, name)


@_on_stream
def pmqa_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                      row_begin, max_rows: int, *, ws=None, stream=None) -> None:
    """Quantise new tokens k, v (bf16 [rows, kv_heads, head_dim]) into the
    cache's blocks, updating the pools and their scales in place."""
    p = make_cache_problem(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                           row_begin, k.shape[0], max_rows)
    dev, bf16, shape = k_cache.get_device(), _torch()[2], (p.rows, p.kv_heads, p.head_dim)
    _like(k, dev, bf16, shape)
    _like(v, dev, bf16, shape)
    _cache_call("pmqa_cache_append", p, dev, stream, ws, k.data_ptr(), v.data_ptr())


@_on_stream
def pmqa_cache_attention(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                         row_begin, max_rows: int, sm_scale: float, *, out=None, lse=None,
                         want_lse: bool = False, ws=None, stream=None):
    """Attention of q (bf16 [rows, heads, head_dim]) to the cached tokens: bf16
    out of q's shape (and fp32 lse [rows, heads] when asked for or given)."""
    import torch

    rows, heads = q.shape[:2]
    p = make_cache_problem(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                           row_begin, rows, max_rows)
    dev = k_cache.get_device()
    f32, _, bf16 = _torch()[:3]
    shape = (rows, heads, p.head_dim)
    _like(q, dev, bf16, shape)
    if out is None:
        out = torch.empty_like(q)
    else:
        _like(out, dev, bf16, shape)
    if lse is None:
        lse = torch.empty((rows, heads), dtype=f32, device=q.device) if want_lse else None
    else:
        _like(lse, dev, f32, (rows, heads))
    _cache_call("pmqa_cache_attention", p, dev, stream, ws, q.data_ptr(), heads, sm_scale,
                out.data_ptr(), None if lse is None else lse.data_ptr())
    return out if lse is None else (out, lse)


@_on_stream
def pmqa_cache_weigh(q, k_cache, k_scale, block_tables, context_lens, row_begin, max_rows: int,
                     sm_scale: float, lse, mass_in=None, *, mass_out=None, mass_width=None,
                     ws=None, stream=None):
    """mass_in (fp32 [bs, kv_heads, mass_width], None for zeros) plus the
    attention weight that each cached token receives from the rows of q, whose
    log-sum-exp `lse` the attention call returned. Only entries of cached tokens
    are written to mass_out (which may be mass_in); a new one starts as a copy
    of mass_in, or as zeros."""
    rows, heads = q.shape[:2]
    p = make_cache_problem(k_cache, None, k_scale, None, block_tables, context_lens, row_begin,
                           rows, max_rows)
    dev = k_cache.get_device()
    f32, _, bf16 = _torch()[:3]
    _like(q, dev, bf16, (rows, heads, p.head_dim))
    _like(lse, dev, f32, (rows, heads))
    given = mass_in if mass_out is None else mass_out
    if given is not None and mass_width not in (None, given.shape[-1]):
        raise AssertionError(f"mass_width {mass_width} beside masses of {given.shape[-1]}")
    width = given.shape[-1] if given is not None else mass_width or p.block_size * p.max_blocks_per_seq
    shape = (p.bs, p.kv_heads, width)
    if mass_in is not None:
        _like(mass_in, dev, f32, shape)
    if mass_out is None:
        mass_out = q.new_zeros(shape, dtype=f32) if mass_in is None else mass_in.clone()
    else:
        _like(mass_out, dev, f32, shape)
    _cache_call("pmqa_cache_weigh", p, dev, stream, ws, q.data_ptr(), heads, sm_scale,
                lse.data_ptr(), None if mass_in is None else mass_in.data_ptr(),
                mass_out.data_ptr(), width)
    return mass_out


@_on_stream
def pmqa_cache_evict(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, mass,
                     keep: int, sinks: int, recent: int, new_tables, *, kept=None, lens_out=None,
                     mass_out=None, ws=None, stream=None):
    """Keep at most `keep` tokens per request and kv head (the first `sinks`,
    the last `recent`, and those with the most mass) in the blocks of
    new_tables; returns (kept [bs, kv_heads, keep], lens_out [bs], mass_out)."""
    import torch

    p = make_cache_problem(k_cache, v_cache, k_scale, v_scale, block_tables, context_lens)
    dev = k_cache.get_device()
    f32, i32 = _torch()[:2]
    width, pairs = mass.shape[-1], (p.bs, p.kv_heads)
    _like(mass, dev, f32, (*pairs, width))
    _like(new_tables, dev, i32, (p.bs, new_tables.shape[-1]))
    if kept is None:
        kept = torch.empty((*pairs, max(keep, 0)), dtype=i32, device=mass.device)
    else:
        _like(kept, dev, i32, (*pairs, keep))
    if lens_out is None:
        lens_out = torch.empty_like(context_lens)
    else:
        _like(lens_out, dev, i32, (p.bs,))
    if mass_out is None:
        mass_out = torch.empty_like(mass)
    else:
        _like(mass_out, dev, f32, (*pairs, width))
    _cache_call("pmqa_cache_evict", p, dev, stream, ws, mass.data_ptr(), width, keep, sinks,
                recent, new_tables.data_ptr(), new_tables.shape[-1], kept.data_ptr(),
                lens_out.data_ptr(), mass_out.data_ptr())
    return kept, lens_out, mass_out


def rope_frequencies(dim: int, base: float = 10000.0, *, kind: int = PMQA_ROPE_PLAIN,
                     factor: float = 1.0, trained: float = 4096.0, slow_turns: float = 1.0,
                     fast_turns: float = 32.0, device=None):
    """Radians per position of the dim / 2 pairs of a rotated head, scaled for contexts
    `factor` times as long as `trained`, as a float64 tensor on the device, and the
    scale that goes with them: what Rotary takes."""
    import torch

    if dim < 2 or dim % 2:
        raise PmqaError(PMQA_ERR_INVALID_ARG, "pmqa_rope_frequencies")
    out, scale = (ctypes.c_double * (dim // 2))(), ctypes.c_float()
    _check(load().pmqa_rope_frequencies(dim, base, kind, factor, trained, slow_turns, fast_turns,
                                        out, ctypes.byref(scale)), "pmqa_rope_frequencies")
    return torch.tensor(list(out), dtype=torch.float64, device=device or "cuda"), scale.value


# The calls below are made once per layer and step, most of them on a few rows: what
# they check and marshal is written out to cost little (a tensor attribute takes about
# 0.1 us, a Python call 0.3, torch.empty 1.7, the launch 2).

def _rotary(rotary, positions, rows: int, dev: int):
    """A pmqa_rotary, or None for none."""
    if rotary is None:
        return None
    names = _torch()
    f, begin, interleaved, scale = rotary
    n = f.numel()
    if f.dtype is not names[6] or f.dim() != 1 or f.get_device() != dev or not f.is_contiguous():
        _like(f, dev, names[6], (n,))
    if positions is not None:
        _like(positions, dev, names[1], (rows,))
        positions = positions.data_ptr()
    return RotaryArgs(f.data_ptr(), positions, 2 * n, begin, 1 if interleaved else 0, scale)


def _norm(norm, width: int, dev: int):
    """A pmqa_norm, or None for none."""
    if norm is None or norm[0] == PMQA_NORM_NONE:
        return None
    kind, weight, bias, eps = norm
    if weight is not None:
        _like(weight, dev, _torch()[0], (width,))
        weight = weight.data_ptr()
    if bias is not None:
        _like(bias, dev, _torch()[0], (width,))
        bias = bias.data_ptr()
    return NormArgs(kind, eps, weight, bias)


def _strided(t, dev: int, shape):
    """The strides of an operand of bf16 rows: on the cache's device, of the documented
    shape, its last dimension contiguous (the others may be strided)."""
    strides = t.stride()
    if t.shape != shape or t.dtype is not _torch()[2] or strides[-1] != 1 or t.get_device() != dev:
        raise AssertionError(f"expected a bfloat16 tensor of shape {tuple(shape)} with a contiguous last "
                             f"dimension on the cache's device ({dev}), got {tuple(t.shape)} {t.dtype} "
                             f"with strides {t.stride()} on {t.device}")
    return strides


def _codes_like(t, dev: int, shape) -> None:
    """A tensor of e4m3 codes."""
    if t.shape != shape or t.dtype not in _torch()[5] or t.get_device() != dev or not t.is_contiguous():
        raise AssertionError(f"expected a contiguous float8_e4m3fn (or uint8) tensor of shape {tuple(shape)} "
                             f"on the cache's device ({dev}), got {tuple(t.shape)} {t.dtype} on {t.device}")


def _device_call(fn, dev: int, stream, *args) -> None:
    """Call a function of the library with device `dev` current, on its current stream
    unless one is given."""
    if dev < 0:
        raise AssertionError(f"{fn.__name__} takes cuda tensors")
    names = _torch()
    if dev != names[3]():
        import torch

        with torch.cuda.device(dev):
            return _device_call(fn, dev, stream, *args)
    rc = fn(*args, names[4](dev) if stream is None else stream.cuda_stream)
    if rc != PMQA_OK:
        raise PmqaError(rc, fn.__name__)


def _paged_call(fn, dev: int, stream, ws, make, *args) -> None:
    """A call that ends with a workspace (`make` makes it unless given) and a stream."""
    if dev < 0:
        raise AssertionError(f"{fn.__name__} takes cuda tensors")
    if ws is None:
        ws = make(f"cuda:{dev}", stream)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise AssertionError("expected a contiguous workspace on the cache's device")
    _device_call(fn, dev, stream, *args, ws.data_ptr(), ws.nbytes)


def _heads(x, dev: int, rows: int, out):
    """A pmqa_heads of x, [rows, heads, head_dim], and its result (a new tensor unless
    given)."""
    _, heads, width = x.shape
    shape = (rows, heads, width)
    xr, xh, _ = _strided(x, dev, shape)
    if out is None:
        out = _torch()[7](shape, dtype=x.dtype, device=x.device)
        return Heads(x.data_ptr(), out.data_ptr(), xr, xh, heads * width, width, heads, width), out
    o_r, oh, _ = _strided(out, dev, shape)
    return Heads(x.data_ptr(), out.data_ptr(), xr, xh, o_r, oh, heads, width), out


@_on_stream
def pmqa_rope(x, positions, rotary: Rotary, *, other=None, out=None, other_out=None, stream=None):
    """Rotate the heads of x (bf16 [rows, heads, head_dim], the last dimension
    contiguous) at positions (int32 [rows]) into `out` (a new tensor unless given; x
    itself rotates in place). `other`: a second tensor of the same rows (the keys
    beside the queries), rotated by the same launch into other_out; then both results
    are returned."""
    fn, rows, dev = (_lib or load()).pmqa_rope, x.shape[0], x.get_device()
    a, out = _heads(x, dev, rows, out)
    r = _rotary(rotary, positions, rows, dev)
    if other is None:
        _device_call(fn, dev, stream, r, rows, a, None)
        return out
    b, other_out = _heads(other, dev, rows, other_out)
    _device_call(fn, dev, stream, r, rows, a, b)
    return out, other_out


def make_paged_rows(kv_cache, width: int, block_tables, context_lens, row_begin, rows: int,
                    max_rows: int) -> PagedRows:
    """Fill a pmqa_paged_rows for a pool [num_blocks, block_size, width] of bytes or
    e4m3 values (context_lens None where the call has none)."""
    names = _torch()
    shape = kv_cache.shape
    if len(shape) != 3 or shape[2] != width or kv_cache.dtype not in names[5] or not kv_cache.is_contiguous():
        raise AssertionError(f"expected a contiguous pool [num_blocks, block_size, {width}] of uint8 or "
                             f"float8_e4m3fn, got {tuple(kv_cache.shape)} {kv_cache.dtype}")
    dev, i32 = kv_cache.get_device(), names[1]
    bs, blocks = block_tables.shape
    _like(block_tables, dev, i32, (bs, blocks))
    if context_lens is not None:
        _like(context_lens, dev, i32, (bs,))
        context_lens = context_lens.data_ptr()
    _like(row_begin, dev, i32, (bs + 1,))
    return PagedRows(block_tables.data_ptr(), context_lens, row_begin.data_ptr(), bs, shape[1], blocks, rows,
                     max_rows, shape[0])


def _status_workspace(device=None, stream=None):
    """The smallest workspace: a status word."""
    import torch

    with torch.cuda.stream(stream):
        ws = torch.empty(256, dtype=torch.uint8, device=device or "cuda")
        with torch.cuda.device(ws.device):
            pmqa_workspace_init(ws, stream=stream)
    return ws


def pmqa_latent_workspace_bytes() -> int:
    return int(load().pmqa_latent_workspace_bytes())


def latent_workspace(device=None, stream=None):
    """A zero-initialised workspace for pmqa_latent_attention (and every other call on
    the indexer's and the latent cache). With a `stream` the memory is that stream's too."""
    import torch

    with torch.cuda.stream(stream):
        ws = torch.empty(pmqa_latent_workspace_bytes(), dtype=torch.uint8, device=device or "cuda")
        with torch.cuda.device(ws.device):
            pmqa_workspace_init(ws, stream=stream)
    return ws


@_on_stream
def pmqa_index_append(k, kv_cache, block_tables, context_lens, row_begin, max_rows: int, *, q=None,
                      weights=None, weight_scale: float = 1.0, norm: Norm | None = None,
                      rotary: Rotary | None = None, positions=None, q_out=None, weights_out=None,
                      ws=None, stream=None):
    """Normalise, rotate and quantise a step's indexer keys k (bf16 [rows, 128], or None)
    into their slots of kv_cache, and its queries q (bf16 [rows, heads, 128]) with their
    head weights (float32 or bfloat16 [rows, heads]) into what the logits calls take:
    returns (q_out fp8 [rows, heads, 128], weights_out float32 [rows, heads]) where q
    is given. positions: int32 [rows], the rows' slots unless given."""
    f32, _, bf16, _, _, codes, _, empty = _torch()
    if k is None and q is None:
        raise AssertionError("expected keys, queries or both")
    rows, dev = (k if q is None else q).shape[0], kv_cache.get_device()
    p = make_paged_rows(kv_cache, 132, block_tables, context_lens, row_begin, rows, max_rows)
    k_addr, k_row = None, 0
    if k is not None:
        k_row = _strided(k, dev, (rows, 128))[0]
        k_addr = k.data_ptr()
    if q is None:
        x = IndexRows(k_addr, None, None, None, None, k_row)
    else:
        heads = q.shape[1]
        shape, pair = (rows, heads, 128), (rows, heads)
        q_row, q_head, _ = _strided(q, dev, shape)
        if weights is None:
            raise AssertionError("expected weights beside q")
        w_row, w_step = weights.stride()
        if weights.shape != pair or weights.dtype not in (f32, bf16) or w_step != 1 and heads > 1 or \
                weights.get_device() != dev:
            raise AssertionError(f"expected float32 or bfloat16 weights of shape {pair} with a "
                                 f"contiguous last dimension, got {tuple(weights.shape)} {weights.dtype}")
        if q_out is None:
            q_out = empty(shape, dtype=codes[0], device=q.device)
        else:
            _codes_like(q_out, dev, shape)
        if weights_out is None:
            weights_out = empty(pair, dtype=f32, device=q.device)
        else:
            _like(weights_out, dev, f32, pair)
        x = IndexRows(k_addr, q.data_ptr(), weights.data_ptr(), q_out.data_ptr(), weights_out.data_ptr(), k_row,
                      q_row, q_head, w_row, heads, 1 if weights.dtype is bf16 else 0, weight_scale)
    _paged_call((_lib or load()).pmqa_index_append, dev, stream, ws, _status_workspace, p, kv_cache.data_ptr(), x,
                _norm(norm, 128, dev), _rotary(rotary, positions, rows, dev))
    return None if q is None else (q_out, weights_out)


@_on_stream
def pmqa_index_read(kv_cache, block_tables, row_begin, rows: int, *, start=None, k=None,
                    k_scale=None, ws=None, stream=None):
    """Cached indexer keys as contiguous rows: row row_begin[i] + j of (k fp8 [rows, 128],
    k_scale float32 [rows]) is the token at slot start[i] + j of request i (start: int32
    [bs], zeros unless given)."""
    f32, i32, _, _, _, codes, _, empty = _torch()
    dev = kv_cache.get_device()
    p = make_paged_rows(kv_cache, 132, block_tables, None, row_begin, rows, 0)
    if start is not None:
        _like(start, dev, i32, (p.bs,))
        start = start.data_ptr()
    if k is None:
        k = empty((max(rows, 0), 128), dtype=codes[0], device=kv_cache.device)
    else:
        _codes_like(k, dev, (rows, 128))
    if k_scale is None:
        k_scale = empty(max(rows, 0), dtype=f32, device=kv_cache.device)
    else:
        _like(k_scale, dev, f32, (rows,))
    _paged_call((_lib or load()).pmqa_index_read, dev, stream, ws, _status_workspace, p, kv_cache.data_ptr(), start,
                k.data_ptr(), k_scale.data_ptr())
    return k, k_scale


@_on_stream
def pmqa_latent_append(c, k_pe, kv_cache, block_tables, context_lens, row_begin, max_rows: int,
                       kv_scale: float, *, q_c=None, q_pe=None, q_scale: float = 1.0,
                       norm: Norm | None = None, rotary: Rotary | None = None, positions=None,
                       q_out=None, ws=None, stream=None):
    """Quantise a step's latent rows (c bf16 [rows, 512], normalised; k_pe bf16
    [rows, 64], rotated; both or neither None) into their slots of the latent cache, and
    its queries (q_c bf16 [rows, heads, 512], q_pe bf16 [rows, heads, 64]) into q_out fp8
    [rows, heads, 576], which is returned where q_c is given."""
    _, _, _, _, _, codes, _, empty = _torch()
    if c is None and q_c is None or (c is None) != (k_pe is None) or (q_c is None) != (q_pe is None):
        raise AssertionError("expected latent rows with their rotary part, queries with theirs, or both")
    rows, dev = (c if q_c is None else q_c).shape[0], kv_cache.get_device()
    p = make_paged_rows(kv_cache, 576, block_tables, context_lens, row_begin, rows, max_rows)
    c_addr, pe_addr, c_row, pe_row = None, None, 0, 0
    if c is not None:
        c_row, pe_row = _strided(c, dev, (rows, 512))[0], _strided(k_pe, dev, (rows, 64))[0]
        c_addr, pe_addr = c.data_ptr(), k_pe.data_ptr()
    if q_c is None:
        x = LatentRows(c_addr, pe_addr, None, None, None, c_row, pe_row, 0, 0, 0, 0, 0, kv_scale, q_scale)
    else:
        heads = q_c.shape[1]
        shape = (rows, heads, 576)
        qc_row, qc_head, _ = _strided(q_c, dev, (rows, heads, 512))
        qp_row, qp_head, _ = _strided(q_pe, dev, (rows, heads, 64))
        if q_out is None:
            q_out = empty(shape, dtype=codes[0], device=q_c.device)
        else:
            _codes_like(q_out, dev, shape)
        x = LatentRows(c_addr, pe_addr, q_c.data_ptr(), q_pe.data_ptr(), q_out.data_ptr(), c_row, pe_row, qc_row,
                       qc_head, qp_row, qp_head, heads, kv_scale, q_scale)
    _paged_call((_lib or load()).pmqa_latent_append, dev, stream, ws, _status_workspace, p, kv_cache.data_ptr(), x,
                _norm(norm, 512, dev), _rotary(rotary, positions, rows, dev))
    return q_out


@_on_stream
def pmqa_latent_attention(q, kv_cache, block_tables, context_lens, row_begin, max_rows: int,
                          q_scale: float, kv_scale: float, sm_scale: float, *, out=None, lse=None,
                          want_lse: bool = False, ws=None, stream=None):
    """Attention of q (fp8 [rows, heads, 576]) to all the latent tokens that its rows
    see: bf16 out [rows, heads, 512] (and float32 lse [rows, heads] when asked for or
    given)."""
    f32, _, bf16, _, _, _, _, empty = _torch()
    rows, heads = q.shape[:2]
    dev, pair = kv_cache.get_device(), (rows, heads)
    p = make_paged_rows(kv_cache, 576, block_tables, context_lens, row_begin, rows, max_rows)
    _codes_like(q, dev, (rows, heads, 576))
    if out is None:
        out = empty((rows, heads, 512), dtype=bf16, device=q.device)
    else:
        _like(out, dev, bf16, (rows, heads, 512))
    if lse is not None:
        _like(lse, dev, f32, pair)
    elif want_lse:
        lse = empty(pair, dtype=f32, device=q.device)
    _paged_call((_lib or load()).pmqa_latent_attention, dev, stream, ws, latent_workspace, p, q.data_ptr(),
                kv_cache.data_ptr(), heads, q_scale, kv_scale, sm_scale, out.data_ptr(),
                None if lse is None else lse.data_ptr())
    return out if lse is None else (out, lse)


def pmqa_gather_probe(pool, rows, row_pitch, method, *, out=None, stream=None):
    """Read the pool's rows `rows` (int32) as 16-byte aligned windows by one
    of three issue methods (a timing aid; include/pmqa.h). Returns `out`
    (uint32 [2] viewed as int32: status bits, XOR of what was read), which
    accumulates over calls when passed in."""
    import torch

    assert rows.dtype == torch.int32 and rows.is_contiguous() and pool.is_contiguous()
    if out is None:
        out = torch.zeros(2, dtype=torch.int32, device=pool.device)
    _check(load().pmqa_gather_probe(_ptr(pool), pool.numel() * pool.element_size(), _ptr(rows),
                                    rows.numel(), row_pitch, method, _ptr(out), _stream(stream)),
           "pmqa_gather_probe")
    return out


def pmqa_read_device_status(ws, stream=None) -> int:
    rc = load().pmqa_read_device_status(_ptr(ws), _stream(stream))
    if rc < 0:
        raise PmqaError(rc, "pmqa_read_device_status")
    return rc


def pmqa_version() -> int:
    return int(load().pmqa_version())
