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
from ._block import _at, _here, _marshal, _raw_stream
from ._lib import _check

EXPORTED_ATTN = (
    "fp8rl_attn_decode",
    "fp8rl_attn_decode_workspace_bytes",
    "fp8rl_kv_read",
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


def declare_attn(L: ctypes.CDLL) -> ctypes.CDLL:
    """Set the argument and result types of these functions on a loaded copy of the library."""
    sz, ci, ptr = ctypes.c_size_t, ctypes.c_int, ctypes.POINTER
    sig = {
        "fp8rl_attn_decode": (ci, [ptr(AttnDecodeArgs), _P, sz, _P]),
        "fp8rl_attn_decode_workspace_bytes": (sz, [_I64, _I32, _I32, _I32, _I64, _I32]),
        "fp8rl_kv_read": (ci, [ptr(KvReadArgs), _P]),
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
