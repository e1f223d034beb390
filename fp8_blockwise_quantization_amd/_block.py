"""Python face of the operators between the FP8 linears (include/fp8rl_block.h).

As in ``_lib``: argument marshalling only, one Python function per C entry point, outputs allocated
where the caller gives none, a non-zero status raised as ``Fp8rlError``. The tensors of a call must
live on one device, which need not be the current one; the call runs there on that device's current
stream, or on ``stream``.

The checks of a call's tensors are compiled (``_marshal``, csrc/marshal.cpp): interpreted, they took
longer than the launch they precede (an append's 22 tensors 8 us, a norm's seven 3 us).
"""

from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from . import _lib
from ._lib import FP8RL_SCALE_FP32, _check, _on_stream, _scale_code
from .build import MARSHAL_PATH

FP8RL_IDS_I32 = 0
FP8RL_IDS_I64 = 1

EXPORTED_BLOCK = (
    "fp8rl_add_rmsnorm_quant",
    "fp8rl_add_rmsnorm_bwd",
    "fp8rl_add_rmsnorm_bwd_workspace_bytes",
    "fp8rl_moe_sort",
    "fp8rl_moe_sort_workspace_bytes",
    "fp8rl_moe_dispatch",
    "fp8rl_moe_combine",
    "fp8rl_moe_combine_bwd",
    "fp8rl_rope_kv_append",
)


class RopeKvArgs(ctypes.Structure):
    """fp8rl_rope_kv_args (include/fp8rl_block.h)."""

    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("ld_q", ctypes.c_int64), ("ld_k", ctypes.c_int64), ("ld_v", ctypes.c_int64),
        ("T", ctypes.c_int64),
        ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
        ("positions", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int64),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p), ("ld_qo", ctypes.c_int64), ("q_scale", ctypes.c_void_p),
        ("slot_mapping", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
        ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
    ]


def declare_block(L: ctypes.CDLL) -> ctypes.CDLL:
    """Set the argument and result types of these functions on a loaded copy of the library."""
    i64, vp, i32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    ci, f32 = ctypes.c_int, ctypes.c_float
    sig = {
        "fp8rl_add_rmsnorm_quant": (ci, [vp, i64, vp, i64, vp, f32, i64, i64, vp, i64, vp, i64, vp,
                                         i64, vp, ci, vp]),
        "fp8rl_add_rmsnorm_bwd": (ci, [vp, i64, vp, i64, vp, vp, i64, f32, i64, i64, vp, i64, vp,
                                       vp, sz, vp]),
        "fp8rl_add_rmsnorm_bwd_workspace_bytes": (sz, [i64, i64]),
        "fp8rl_moe_sort": (ci, [vp, ci, i64, i32, i32, vp, vp, vp, vp, sz, vp]),
        "fp8rl_moe_sort_workspace_bytes": (sz, [i64, i32, i32]),
        "fp8rl_moe_dispatch": (ci, [vp, i64, vp, i64, i32, i64, vp, i64, i64, vp]),
        "fp8rl_moe_combine": (ci, [vp, ci, i64, i64, vp, vp, i64, i32, i64, vp, ci, i64, vp]),
        "fp8rl_moe_combine_bwd": (ci, [vp, i64, vp, i64, ci, i64, vp, vp, i64, i32, i64, vp, i64,
                                       vp, vp]),
        "fp8rl_rope_kv_append": (ci, [ctypes.POINTER(RopeKvArgs), vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


_L = None


def _block_lib() -> ctypes.CDLL:
    global _L
    if _L is None:
        _L = declare_block(_lib.lib())
    return _L


_m = None


def _marshal():
    """The compiled marshalling module, loaded once."""
    global _m
    if _m is None:
        _lib.lib()  # raises where nothing is built
        try:
            from . import _marshal as module
        except ImportError as e:
            what = (f"cannot be loaded ({e}); build it again with the torch that is installed"
                    if os.path.exists(MARSHAL_PATH) else "is not built")
            raise RuntimeError(f"the argument marshalling {what}: run "
                               "`python -m fp8_blockwise_quantization_amd.build`") from e
        _m = module
    return _m


@contextlib.contextmanager
def _at(t, name, stream):
    """Make t's device current and, where `stream` is given, that stream torch's current one (so
    that what the call allocates belongs to it)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device (cuda) tensor")
    with torch.cuda.device(t.get_device()), _on_stream(stream):
        if torch.cuda.current_device() != t.get_device():
            raise ValueError(f"stream belongs to another device than {name}")
        yield


def _here(t, stream) -> int:
    """The device of a call's first tensor where the call can run as things stand; else -1 (a
    stream was given, or the device is not the current one, or t is no device tensor)."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    return dev if stream is None and dev >= 0 and dev == torch._C._cuda_getDevice() else -1


# The address of the device's current stream in torch (`stream` itself under _at).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (none without a GPU build)


def _shape2(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.shape


# ------------------------------------------------------------------------------------------ norm


def fp8rl_add_rmsnorm_quant(x, weight, residual=None, eps=1e-6, h=None, y=None, xq=None, sa=None,
                            rows: bool = False, codes: bool = True, scale="fp32", stream=None):
    """Residual addition, root-mean-square norm and 1x128 quantization of bf16 x [M][K].

    Returns (xq, sa, h, y): uint8 codes [M][K] and float32 scales [M][K/128] of the normalised
    rows (None with ``codes=False``), the bf16 stream h = x + residual (None without ``residual``)
    and the bf16 normalised rows y (with ``rows=True`` or a tensor ``y``; else None). ``h`` may be
    ``x`` or ``residual`` itself. ``scale`` is 'fp32' or 'pow2'."""
    dev = _here(x, stream)
    if dev < 0:
        with _at(x, "x", stream):
            return fp8rl_add_rmsnorm_quant(x, weight, residual, eps, h, y, xq, sa, rows, codes,
                                           scale)
    if residual is not None and h is None:
        h = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    if rows and y is None:
        y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    if xq is None or sa is None:
        if codes or xq is not None or sa is not None:
            M, K = _shape2(x, "x")
            if xq is None:
                xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
            if sa is None:
                sa = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
    fmt = FP8RL_SCALE_FP32 if scale == "fp32" else _scale_code(scale)
    _check((_m or _marshal()).add_rmsnorm_quant(x, weight, residual, eps, h, y, xq, sa, fmt, dev,
                                                _raw_stream(dev)), "fp8rl_add_rmsnorm_quant")
    return xq, sa, h, y


def fp8rl_add_rmsnorm_bwd_workspace_bytes(M: int, K: int) -> int:
    return int(_block_lib().fp8rl_add_rmsnorm_bwd_workspace_bytes(M, K))


def fp8rl_add_rmsnorm_bwd(dy, h, weight, dh=None, eps=1e-6, dx=None, dw=None,
                          weight_grad: bool = True, workspace=None, stream=None):
    """Backward pass of the norm: (dx, dw) from the gradient dy at its output, the stream h it was
    taken of and, if any, the gradient dh that reaches the stream from behind. dx (bf16 [M][K]) is
    the gradient of x and of residual; it may be written in place of dy or dh. dw is float32 [K]
    (None with ``weight_grad=False``)."""
    dev = _here(dy, stream)
    if dev < 0:
        with _at(dy, "dy", stream):
            return fp8rl_add_rmsnorm_bwd(dy, h, weight, dh, eps, dx, dw, weight_grad, workspace)
    if dx is None:
        dx = torch.empty(dy.shape, dtype=torch.bfloat16, device=dy.device)
    if dw is None and weight_grad:
        dw = torch.empty(_shape2(dy, "dy")[1], dtype=torch.float32, device=dy.device)
    _check((_m or _marshal()).add_rmsnorm_bwd(dy, h, weight, dh, eps, dx, dw, workspace, dev,
                                              _raw_stream(dev)), "fp8rl_add_rmsnorm_bwd")
    return dx, dw


# --------------------------------------------------------------------------------------- experts


def fp8rl_moe_sort_workspace_bytes(T: int, top_k: int, E: int) -> int:
    return int(_block_lib().fp8rl_moe_sort_workspace_bytes(T, top_k, E))


def fp8rl_moe_sort(topk_ids, E: int, expert_offsets=None, row_ids=None, pos=None, workspace=None,
                   stream=None):
    """The router's choices topk_ids [T][top_k] (int32 or int64, contiguous; an id outside [0, E)
    is another rank's) in expert order: int32 (expert_offsets [E + 1], row_ids [T * top_k],
    pos [T][top_k]). expert_offsets and row_ids are what the grouped GEMMs read; pos is the grouped
    row of each choice, -1 where it has none."""
    dev = _here(topk_ids, stream)
    if dev < 0:
        with _at(topk_ids, "topk_ids", stream):
            return fp8rl_moe_sort(topk_ids, E, expert_offsets, row_ids, pos, workspace)
    if expert_offsets is None:
        expert_offsets = torch.empty(max(E, 0) + 1, dtype=torch.int32, device=topk_ids.device)
    if row_ids is None:
        row_ids = torch.empty(topk_ids.numel(), dtype=torch.int32, device=topk_ids.device)
    if pos is None:
        pos = torch.empty(topk_ids.shape, dtype=torch.int32, device=topk_ids.device)
    _check((_m or _marshal()).moe_sort(topk_ids, E, expert_offsets, row_ids, pos, workspace, dev,
                                       _raw_stream(dev)), "fp8rl_moe_sort")
    return expert_offsets, row_ids, pos


def fp8rl_moe_dispatch(x, pos, out=None, stream=None):
    """Token rows moved into expert order: out[pos[t][j]] = x[t]. ``out`` (bf16 [R][N]) is
    allocated with a row per choice when not given; rows that no choice names are not written."""
    dev = _here(x, stream)
    if dev < 0:
        with _at(x, "x", stream):
            return fp8rl_moe_dispatch(x, pos, out)
    if out is None:
        out = torch.empty((pos.numel(), _shape2(x, "x")[1]), dtype=torch.bfloat16, device=x.device)
    _check((_m or _marshal()).moe_dispatch(x, pos, out, dev, _raw_stream(dev)),
           "fp8rl_moe_dispatch")
    return out


def fp8rl_moe_combine(y, pos, weights=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """out[t] = sum over j of weights[t][j] * y[pos[t][j]] (bf16 or float32 y [R][N], float32
    weights [T][top_k] or None for ones); choices without a row (pos < 0) add nothing."""
    dev = _here(y, stream)
    if dev < 0:
        with _at(y, "y", stream):
            return fp8rl_moe_combine(y, pos, weights, out_dtype, out)
    if out is None:
        out = torch.empty((_shape2(pos, "pos")[0], _shape2(y, "y")[1]), dtype=out_dtype,
                          device=y.device)
    _check((_m or _marshal()).moe_combine(y, pos, weights, out, dev, _raw_stream(dev)),
           "fp8rl_moe_combine")
    return out


def fp8rl_moe_combine_bwd(dout, y, pos, weights=None, dy=None, dweights=None, R=None,
                          y_dtype=torch.bfloat16, stream=None):
    """Gradients of fp8rl_moe_combine: (dy, dweights) from bf16 dout [T][N]. dy[pos[t][j]] =
    weights[t][j] * dout[t] in y's type (rows that no choice names are not written); dweights
    float32 [T][top_k]. With ``y=None`` only dy is formed, [R][N] of ``y_dtype`` (R: a row per
    choice unless given). dy may be written in place of y."""
    dev = _here(dout, stream)
    if dev < 0:
        with _at(dout, "dout", stream):
            return fp8rl_moe_combine_bwd(dout, y, pos, weights, dy, dweights, R, y_dtype)
    if y is not None:
        if dweights is None:
            dweights = torch.empty(pos.shape, dtype=torch.float32, device=dout.device)
        if dy is None:
            dy = torch.empty(y.shape, dtype=y.dtype, device=dout.device)
    elif dweights is not None:
        raise ValueError("dweights needs y")
    elif dy is None:
        dy = torch.empty((pos.numel() if R is None else R, _shape2(dout, "dout")[1]),
                         dtype=y_dtype, device=dout.device)
    _check((_m or _marshal()).moe_combine_bwd(dout, y, pos, weights, dy, dweights, dev,
                                              _raw_stream(dev)), "fp8rl_moe_combine_bwd")
    return dy, dweights


# -------------------------------------------------------------------------------------- KV cache


def fp8rl_rope_kv_append(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_out=None,
                         interleaved: bool = False, q_weight=None, k_weight=None, eps=1e-6,
                         q_scale=None, k_scale=None, v_scale=None, stream=None):
    """Rotate q and k by their positions (after per-head norms where ``q_weight`` and ``k_weight``,
    bf16 [D], are given) and store k and v into a paged cache; returns the rotated q.

    q [T][Hq * D], k and v [T][Hkv * D] are bf16 rows, e.g. column slices of one fused output.
    ``cos_sin`` float32 [max_pos][rot_dim] holds the cosines, then the sines, of each position's
    angles; ``positions`` and ``slot_mapping`` are int64 [T]. The caches are 4-D views
    [page][place in the page][head][D], alike in shape and strides (``.transpose(1, 2)`` of a cache
    laid out head by head): bf16, or uint8 for E4M3 codes with device scalars ``k_scale`` and
    ``v_scale``. A token with a negative slot stores nothing. ``q_out`` is bf16 (it may be q), or
    uint8 codes with ``q_scale``; q may be None (k and v alone). ``cos_sin`` None rotates nothing."""
    dev = _here(k, stream)
    if dev < 0:
        with _at(k, "k", stream):
            return fp8rl_rope_kv_append(
                q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_out, interleaved,
                q_weight, k_weight, eps, q_scale, k_scale, v_scale)
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=torch.bfloat16 if q_scale is None else torch.uint8,
                            device=k.device)
    _check((_m or _marshal()).rope_kv_append(
        q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_out, interleaved, q_weight,
        k_weight, eps, q_scale, k_scale, v_scale, dev, _raw_stream(dev)), "fp8rl_rope_kv_append")
    return q_out
