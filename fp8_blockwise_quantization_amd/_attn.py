"""Python face of attention (include/fp8rl_attn.h).

As in ``_block``: argument marshalling only, one Python function per C entry point, outputs allocated
where the caller gives none, a non-zero status raised as ``Fp8rlError``; a call runs on its tensors'
device, on that device's current stream or on ``stream``.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._block import _at, _here, _marshal, _raw_stream, _shape2
from ._lib import _check

EXPORTED_ATTN = (
    "fp8rl_attn_decode",
    "fp8rl_attn_decode_workspace_bytes",
    "fp8rl_kv_read",
    "fp8rl_attn_fwd",
    "fp8rl_attn_bwd",
    "fp8rl_attn_bwd_workspace_bytes",
)


class _Args(ctypes.Structure):
    """A host struct of the C ABI, its fields named as there, a type's names in one line."""

    @staticmethod
    def fields(*groups):
        return [(name, kind) for names, kind in groups for name in names.split()]


_P, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class AttnDecodeArgs(_Args):
    """fp8rl_attn_decode_args."""

    _fields_ = _Args.fields(
        ("q", _P), ("ld_q", _I64), ("q_scale", _P), ("B", _I64), ("q_heads kv_heads head_dim", _I32),
        ("k_cache v_cache k_scale v_scale", _P), ("num_pages", _I64), ("page_size", _I32),
        ("page_stride slot_stride head_stride", _I64), ("page_table", _P), ("ld_table", _I64),
        ("table_width", _I32), ("lengths", _P), ("sm_scale", _F32), ("window", _I32), ("cap", _F32),
        ("slopes out", _P), ("ld_out", _I64))


class KvReadArgs(_Args):
    """fp8rl_kv_read_args."""

    _fields_ = _Args.fields(
        ("k_cache v_cache k_scale v_scale", _P), ("num_pages", _I64), ("page_size", _I32),
        ("page_stride slot_stride head_stride", _I64), ("kv_heads head_dim", _I32),
        ("page_table", _P), ("ld_table", _I64), ("table_width", _I32), ("B", _I64),
        ("offsets starts", _P), ("R", _I64), ("k_out v_out", _P), ("ld_k ld_v", _I64))


class AttnArgs(_Args):
    """fp8rl_attn_args."""

    _fields_ = _Args.fields(
        ("q k v", _P), ("ld_q ld_k ld_v Tq Tk", _I64), ("q_heads kv_heads head_dim", _I32),
        ("docs", _I64), ("q_offsets k_offsets", _P), ("causal window", _I32), ("prefix", _P),
        ("sm_scale cap", _F32), ("slopes out", _P), ("ld_out", _I64), ("lse dout", _P),
        ("ld_dout", _I64), ("dq dk dv", _P), ("ld_dq ld_dk ld_dv", _I64))


def declare_attn(L: ctypes.CDLL) -> ctypes.CDLL:
    """Set the argument and result types of these functions on a loaded copy of the library."""
    sz, ci, ptr = ctypes.c_size_t, ctypes.c_int, ctypes.POINTER
    sig = {
        "fp8rl_attn_decode": (ci, [ptr(AttnDecodeArgs), _P, sz, _P]),
        "fp8rl_attn_decode_workspace_bytes": (sz, [_I64, _I32, _I32, _I32, _I64, _I32]),
        "fp8rl_kv_read": (ci, [ptr(KvReadArgs), _P]),
        "fp8rl_attn_fwd": (ci, [ptr(AttnArgs), _P]),
        "fp8rl_attn_bwd": (ci, [ptr(AttnArgs), _P, sz, _P]),
        "fp8rl_attn_bwd_workspace_bytes": (sz, [_I64, _I64, _I64, _I32, _I32, _I32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


_L = None


def _attn_lib() -> ctypes.CDLL:
    global _L
    if _L is None:
        _L = declare_attn(_lib.lib())
    return _L


def fp8rl_attn_decode_workspace_bytes(B: int, q_heads: int, kv_heads: int, head_dim: int,
                                      max_keys: int, window: int = 0) -> int:
    return int(_attn_lib().fp8rl_attn_decode_workspace_bytes(B, q_heads, kv_heads, head_dim,
                                                             max_keys, window))


def fp8rl_attn_decode(q, k_cache, v_cache, page_table, lengths, sm_scale=None, window: int = 0,
                      cap: float = 0.0, slopes=None, q_scale=None, k_scale=None, v_scale=None,
                      out=None, workspace=None, stream=None):
    """Attention of one new token of every sequence over the paged cache: bf16 [B][Hq * D].

    q is bf16 [B][Hq * D], or uint8 codes with the device scalar ``q_scale``, as rope_kv_append
    returns it; the caches are 4-D views [page][place in the page][head][D] as it fills them (bf16, or
    uint8 codes with ``k_scale`` and ``v_scale``). ``page_table`` int32 [B][n] names the pages of each
    sequence, ``lengths`` int32 [B] its cached keys, the new token's included. ``sm_scale`` is
    1 / sqrt(D) unless given. ``window`` keys are seen at most, ``cap`` bounds the scores by
    cap * tanh(s / cap), ``slopes`` float32 [Hq] takes slope * distance off them. A sequence of length
    0 gives zeros."""
    dev = _here(q, stream)
    if dev < 0:
        with _at(q, "q", stream):
            return fp8rl_attn_decode(q, k_cache, v_cache, page_table, lengths, sm_scale, window, cap,
                                     slopes, q_scale, k_scale, v_scale, out, workspace)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if sm_scale is None:
        sm_scale = 1 / math.sqrt(max(k_cache.shape[-1], 1))
    _check(_marshal().attn_decode(q, k_cache, v_cache, page_table, lengths, sm_scale, window, cap,
                                  slopes, q_scale, k_scale, v_scale, out, workspace, dev,
                                  _raw_stream(dev)), "fp8rl_attn_decode")
    return out


def fp8rl_kv_read(k_cache, v_cache, page_table, offsets, starts=None, k_scale=None, v_scale=None,
                  k_out=None, v_out=None, rows=None, stream=None):
    """Cached keys and values back as contiguous rows: (k_out, v_out), bf16 [R][Hkv * D].

    Rows offsets[b] .. offsets[b + 1] - 1 (int32 [B + 1], on the device) are sequence b's keys from
    starts[b] on (int32 [B]; None: from 0). Caches, scales and ``page_table`` are attn_decode's. Rows
    of no sequence are not written; ``rows`` is R where the outputs are not given."""
    dev = _here(k_cache, stream)
    if dev < 0:
        with _at(k_cache, "k_cache", stream):
            return fp8rl_kv_read(k_cache, v_cache, page_table, offsets, starts, k_scale, v_scale,
                                 k_out, v_out, rows)
    if k_out is None or v_out is None:
        if rows is None:
            given = k_out if k_out is not None else v_out
            if given is None:
                raise ValueError("rows is needed where no output is given")
            rows = given.shape[0]
        if k_cache.dim() != 4:
            raise ValueError("k_cache must be 4-D: [page][place][head][column]")
        shape = (rows, k_cache.shape[2] * k_cache.shape[3])
        if k_out is None:
            k_out = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
        if v_out is None:
            v_out = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
    _check(_marshal().kv_read(k_cache, v_cache, page_table, offsets, starts, k_scale, v_scale, k_out,
                              v_out, dev, _raw_stream(dev)), "fp8rl_kv_read")
    return k_out, v_out


def fp8rl_attn_fwd(q, k, v, head_dim: int, q_offsets, k_offsets=None, causal: bool = True,
                   sm_scale=None, window: int = 0, prefix=None, cap: float = 0.0, slopes=None,
                   out=None, lse=None, stream=None):
    """Attention of packed documents: (out, lse), bf16 [Tq][Hq * D] and float32 [Hq][Tq].

    q [Tq][Hq * D], k and v [Tk][Hkv * D] are bf16 rows, e.g. column slices of one fused output;
    document d's queries are rows q_offsets[d] .. q_offsets[d + 1] - 1 (int32, on the device), its keys
    those of ``k_offsets`` (None: the same rows). With Lq queries and Lk keys query i is at position
    p = i + Lk - Lq, and sees key j if (not causal or j <= p) and (no window or p - j < window), or
    if j < prefix[d] (int32 [docs]). ``sm_scale`` is 1 / sqrt(D) unless given; ``cap`` bounds the
    scores by cap * tanh(s / cap), ``slopes`` float32 [Hq] takes slope * |p - j| off them. Rows of no
    document are not written. lse is the log of a query's sum of exponentials, -inf (and zeros in
    out) where it sees no key."""
    dev = _here(q, stream)
    if dev < 0:
        with _at(q, "q", stream):
            return fp8rl_attn_fwd(q, k, v, head_dim, q_offsets, k_offsets, causal, sm_scale, window,
                                  prefix, cap, slopes, out, lse)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        Tq, cols = _shape2(q, "q")
        lse = torch.empty((cols // max(head_dim, 1), Tq), dtype=torch.float32, device=q.device)
    if sm_scale is None:
        sm_scale = 1 / math.sqrt(max(head_dim, 1))
    _check(_marshal().attn_fwd(q, k, v, head_dim, q_offsets, k_offsets, causal, sm_scale, window,
                               prefix, cap, slopes, out, lse, dev, _raw_stream(dev)),
           "fp8rl_attn_fwd")
    return out, lse


def fp8rl_attn_bwd_workspace_bytes(Tq: int, Tk: int, docs: int, q_heads: int, kv_heads: int,
                                   head_dim: int) -> int:
    return int(_attn_lib().fp8rl_attn_bwd_workspace_bytes(Tq, Tk, docs, q_heads, kv_heads, head_dim))


def fp8rl_attn_bwd(dout, q, k, v, out, lse, head_dim: int, q_offsets, k_offsets=None,
                   causal: bool = True, sm_scale=None, window: int = 0, prefix=None, cap: float = 0.0,
                   slopes=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of fp8rl_attn_fwd: (dq, dk, dv), bf16, shaped as q, k and v, from the gradient dout
    at its output and what it returned; the other arguments are that call's. The gradients may be
    column slices of one fused row. Rows of no document are not written."""
    dev = _here(dout, stream)
    if dev < 0:
        with _at(dout, "dout", stream):
            return fp8rl_attn_bwd(dout, q, k, v, out, lse, head_dim, q_offsets, k_offsets, causal,
                                  sm_scale, window, prefix, cap, slopes, dq, dk, dv, workspace)
    if dq is None:
        dq = torch.empty(q.shape, dtype=torch.bfloat16, device=dout.device)
    if dk is None:
        dk = torch.empty(k.shape, dtype=torch.bfloat16, device=dout.device)
    if dv is None:
        dv = torch.empty(v.shape, dtype=torch.bfloat16, device=dout.device)
    if sm_scale is None:
        sm_scale = 1 / math.sqrt(max(head_dim, 1))
    _check(_marshal().attn_bwd(q, k, v, head_dim, q_offsets, k_offsets, causal, sm_scale, window,
                               prefix, cap, slopes, out, lse, dout, dq, dk, dv, workspace, dev,
                               _raw_stream(dev)), "fp8rl_attn_bwd")
    return dq, dk, dv
