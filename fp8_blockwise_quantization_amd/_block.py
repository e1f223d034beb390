"""ctypes binding of the operators between the FP8 linears (include/fp8rl_block.h).

As in ``_lib``: argument marshalling only, one Python function per C entry point, outputs allocated
where the caller gives none, a non-zero status raised as ``Fp8rlError``. The tensors of a call must
live on one device, which need not be the current one; the call runs there on that device's current
stream, or on ``stream``.
"""

from __future__ import annotations

import contextlib
import ctypes
import struct

import torch

from . import _lib
from ._lib import FP8RL_OUT_BF16, FP8RL_OUT_F32, FP8RL_SCALE_FP32, _check, _on_stream, _scale_code

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
        "fp8rl_rope_kv_append": (ci, [vp, vp]),  # the struct by reference or as its bytes
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


# RopeKvArgs as struct.pack lays it out (native alignment, like the C struct): filling bytes costs a
# fraction of filling a ctypes structure.
_pack_rope = struct.Struct("@PPPqqqqiiiiifPPqPPPqPPPPPPqiqqq").pack

_L = None


def _block_lib() -> ctypes.CDLL:
    global _L
    if _L is None:
        _L = declare_block(_lib.lib())
    return _L


_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None


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
    return dev if stream is None and dev >= 0 and dev == _device() else -1


# The address of the device's current stream in torch (`stream` itself under _at).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _fail(name, t, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device (cuda) tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call runs on cuda:{dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be dense along its last dimension (and contiguous where it is "
                     "no matrix of rows)")


def _matrix(t, name, dtype, shape, dev):
    """(address, row pitch) of a [rows][cols] matrix with unit column stride."""
    try:
        stride = t.stride()
        if (t.dtype is dtype and t.get_device() == dev and t.shape == shape
                and (stride[1] == 1 or shape[1] <= 1)):
            return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1]
    except AttributeError:  # no tensor
        pass
    _fail(name, t, dtype, shape, dev)


def _vector(t, name, dtype, shape, dev):
    """Address of a contiguous tensor."""
    try:
        if (t.dtype is dtype and t.get_device() == dev and t.shape == shape
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _fail(name, t, dtype, shape, dev)


def _flat(t, name, dtype, n, dev):
    """Address of a contiguous tensor of n values."""
    try:
        if (t.dtype is dtype and t.get_device() == dev and t.numel() == n
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _fail(name, t, dtype, (n,), dev)


def _workspace(workspace, need, t, dev):
    """(tensor to keep alive, address, bytes) of a call's workspace, allocated beside t if none is
    given."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = t.new_empty(need, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), need
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _out_type(t, name):
    if t.dtype == torch.bfloat16:
        return FP8RL_OUT_BF16
    if t.dtype == torch.float32:
        return FP8RL_OUT_F32
    raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")


def _is_2d(t, name):
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
    bf16 = torch.bfloat16
    M, K = _is_2d(x, "x")
    px, ld_x = _matrix(x, "x", bf16, (M, K), dev)
    pw = _flat(weight, "weight", bf16, K, dev)
    pr = ph = py = pq = ps = None
    ld_r = ld_h = ld_y = ld_q = 0
    if residual is not None:
        pr, ld_r = _matrix(residual, "residual", bf16, (M, K), dev)
        if h is None:
            h = torch.empty((M, K), dtype=bf16, device=x.device)
    if h is not None:
        ph, ld_h = _matrix(h, "h", bf16, (M, K), dev)
    if rows and y is None:
        y = torch.empty((M, K), dtype=bf16, device=x.device)
    if y is not None:
        py, ld_y = _matrix(y, "y", bf16, (M, K), dev)
    if codes or xq is not None or sa is not None:
        if xq is None:
            xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
        if sa is None:
            sa = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
        pq, ld_q = _matrix(xq, "xq", torch.uint8, (M, K), dev)
        ps = _vector(sa, "sa", torch.float32, (M, K // 128), dev)
    fmt = FP8RL_SCALE_FP32 if scale == "fp32" else _scale_code(scale)
    _check(_block_lib().fp8rl_add_rmsnorm_quant(px, ld_x, pr, ld_r, pw, eps, M, K, ph, ld_h, py,
                                                ld_y, pq, ld_q, ps, fmt, _raw_stream(dev)),
           "fp8rl_add_rmsnorm_quant")
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
    bf16 = torch.bfloat16
    M, K = _is_2d(dy, "dy")
    pg, ld_g = _matrix(dy, "dy", bf16, (M, K), dev)
    ph, ld_h = _matrix(h, "h", bf16, (M, K), dev)
    pw = _flat(weight, "weight", bf16, K, dev)
    pd, ld_d = _matrix(dh, "dh", bf16, (M, K), dev) if dh is not None else (None, 0)
    if dx is None:
        dx = torch.empty((M, K), dtype=bf16, device=dy.device)
    px, ld_x = _matrix(dx, "dx", bf16, (M, K), dev)
    if dw is None and weight_grad:
        dw = torch.empty(K, dtype=torch.float32, device=dy.device)
    po = _flat(dw, "dw", torch.float32, K, dev) if dw is not None else None
    L = _block_lib()
    need = L.fp8rl_add_rmsnorm_bwd_workspace_bytes(M, K) if dw is not None else 0
    keep, ws, nbytes = _workspace(workspace, need, dy, dev)
    _check(L.fp8rl_add_rmsnorm_bwd(pg, ld_g, ph, ld_h, pw, pd, ld_d, eps, M, K, px, ld_x, po, ws,
                                   nbytes, _raw_stream(dev)), "fp8rl_add_rmsnorm_bwd")
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
    T, k = _is_2d(topk_ids, "topk_ids")
    if topk_ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"topk_ids must be torch.int32 or torch.int64, got {topk_ids.dtype}")
    i32, device = torch.int32, topk_ids.device
    pi = _vector(topk_ids, "topk_ids", topk_ids.dtype, (T, k), dev)
    if expert_offsets is None:
        expert_offsets = torch.empty(E + 1, dtype=i32, device=device)
    if row_ids is None:
        row_ids = torch.empty(T * k, dtype=i32, device=device)
    if pos is None:
        pos = torch.empty((T, k), dtype=i32, device=device)
    po = _flat(expert_offsets, "expert_offsets", i32, E + 1, dev)
    pr = _flat(row_ids, "row_ids", i32, T * k, dev)
    pp = _vector(pos, "pos", i32, (T, k), dev)
    L = _block_lib()
    keep, ws, nbytes = _workspace(workspace, L.fp8rl_moe_sort_workspace_bytes(T, k, E), topk_ids,
                                  dev)
    wide = FP8RL_IDS_I64 if topk_ids.dtype == torch.int64 else FP8RL_IDS_I32
    _check(L.fp8rl_moe_sort(pi, wide, T, k, E, po, pr, pp, ws, nbytes, _raw_stream(dev)),
           "fp8rl_moe_sort")
    return expert_offsets, row_ids, pos


def fp8rl_moe_dispatch(x, pos, out=None, stream=None):
    """Token rows moved into expert order: out[pos[t][j]] = x[t]. ``out`` (bf16 [R][N]) is
    allocated with a row per choice when not given; rows that no choice names are not written."""
    dev = _here(x, stream)
    if dev < 0:
        with _at(x, "x", stream):
            return fp8rl_moe_dispatch(x, pos, out)
    T, N = _is_2d(x, "x")
    k = _is_2d(pos, "pos")[1]
    px, ld_x = _matrix(x, "x", torch.bfloat16, (T, N), dev)
    pp = _vector(pos, "pos", torch.int32, (T, k), dev)
    if out is None:
        out = torch.empty((T * k, N), dtype=torch.bfloat16, device=x.device)
    R = _is_2d(out, "out")[0]
    po, ld_o = _matrix(out, "out", torch.bfloat16, (R, N), dev)
    _check(_block_lib().fp8rl_moe_dispatch(px, ld_x, pp, T, k, N, po, R, ld_o, _raw_stream(dev)),
           "fp8rl_moe_dispatch")
    return out


def fp8rl_moe_combine(y, pos, weights=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """out[t] = sum over j of weights[t][j] * y[pos[t][j]] (bf16 or float32 y [R][N], float32
    weights [T][top_k] or None for ones); choices without a row (pos < 0) add nothing."""
    dev = _here(y, stream)
    if dev < 0:
        with _at(y, "y", stream):
            return fp8rl_moe_combine(y, pos, weights, out_dtype, out)
    R, N = _is_2d(y, "y")
    T, k = _is_2d(pos, "pos")
    kind = _out_type(y, "y")
    py, ld_y = _matrix(y, "y", y.dtype, (R, N), dev)
    pp = _vector(pos, "pos", torch.int32, (T, k), dev)
    pw = _vector(weights, "weights", torch.float32, (T, k), dev) if weights is not None else None
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=y.device)
    out_kind = _out_type(out, "out")
    po, ld_o = _matrix(out, "out", out.dtype, (T, N), dev)
    _check(_block_lib().fp8rl_moe_combine(py, kind, R, ld_y, pp, pw, T, k, N, po, out_kind, ld_o,
                                          _raw_stream(dev)), "fp8rl_moe_combine")
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
    T, N = _is_2d(dout, "dout")
    k = _is_2d(pos, "pos")[1]
    pg, ld_g = _matrix(dout, "dout", torch.bfloat16, (T, N), dev)
    pp = _vector(pos, "pos", torch.int32, (T, k), dev)
    pw = _vector(weights, "weights", torch.float32, (T, k), dev) if weights is not None else None
    py = pd = None
    ld_y = 0
    if y is not None:
        R, y_dtype = _is_2d(y, "y")[0], y.dtype
        py, ld_y = _matrix(y, "y", y_dtype, (R, N), dev)
        if dweights is None:
            dweights = torch.empty((T, k), dtype=torch.float32, device=dout.device)
        pd = _vector(dweights, "dweights", torch.float32, (T, k), dev)
    elif dweights is not None:
        raise ValueError("dweights needs y")
    if dy is None:
        dy = torch.empty((T * k if R is None else R, N), dtype=y_dtype, device=dout.device)
    elif y is None:
        R, y_dtype = _is_2d(dy, "dy")[0], dy.dtype
    R = dy.shape[0] if R is None else R
    kind = _out_type(dy, "dy")
    po, ld_o = _matrix(dy, "dy", y_dtype, (R, N), dev)
    _check(_block_lib().fp8rl_moe_combine_bwd(pg, ld_g, py, ld_y, kind, R, pp, pw, T, k, N, po,
                                              ld_o, pd, _raw_stream(dev)), "fp8rl_moe_combine_bwd")
    return dy, dweights


# -------------------------------------------------------------------------------------- KV cache


def _cache(t, name, dtype, shape, strides, dev):
    """Address of a cache view of the first one's shape and strides."""
    try:
        if (t.dtype is dtype and t.get_device() == dev and t.shape == shape
                and (strides[3] == 1 or shape[3] <= 1)):
            if t.stride() != strides and shape[0] > 0:
                raise ValueError("k_cache and v_cache must have the same strides")
            return t.data_ptr()
    except AttributeError:
        pass
    _fail(name, t, dtype, shape, dev)


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
    bf16 = torch.bfloat16
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be 4-D: [page][place][head][column]")
    pages, page, Hkv, D = k_cache.shape
    T = _is_2d(k, "k")[0]
    pk, ld_k = _matrix(k, "k", bf16, (T, Hkv * D), dev)
    pv, ld_v = _matrix(v, "v", bf16, (T, Hkv * D), dev)
    kind = bf16 if k_scale is None else torch.uint8
    strides = k_cache.stride()
    pkc = _cache(k_cache, "k_cache", kind, k_cache.shape, strides, dev)
    pvc = _cache(v_cache, "v_cache", kind, k_cache.shape, strides, dev)
    # a dimension of one entry has no stride to speak of
    page_stride = strides[0] if pages > 1 else 0
    slot_stride = strides[1] if page > 1 else D
    head_stride = strides[2] if Hkv > 1 else D
    pq = po = ld_q = ld_o = Hq = 0
    if q is not None:
        cols = _is_2d(q, "q")[1]
        if D == 0 or cols % D:
            raise ValueError(f"q has {cols} columns, no multiple of the head width {D}")
        Hq = cols // D
        pq, ld_q = _matrix(q, "q", bf16, (T, cols), dev)
        q_kind = bf16 if q_scale is None else torch.uint8
        if q_out is None:
            q_out = torch.empty((T, cols), dtype=q_kind, device=k.device)
        po, ld_o = _matrix(q_out, "q_out", q_kind, (T, cols), dev)
    rot = max_pos = pc = pp = qw = kw = qs = ks = vs = 0
    if cos_sin is not None:
        max_pos, rot = _is_2d(cos_sin, "cos_sin")
        pc = _vector(cos_sin, "cos_sin", torch.float32, (max_pos, rot), dev)
        pp = _flat(positions, "positions", torch.int64, T, dev)
    ps = _flat(slot_mapping, "slot_mapping", torch.int64, T, dev)
    if q_weight is not None:
        qw = _flat(q_weight, "q_weight", bf16, D, dev)
    if k_weight is not None:
        kw = _flat(k_weight, "k_weight", bf16, D, dev)
    if q_scale is not None:
        qs = _flat(q_scale, "q_scale", torch.float32, 1, dev)
    if k_scale is not None:
        ks = _flat(k_scale, "k_scale", torch.float32, 1, dev)
    if v_scale is not None:
        vs = _flat(v_scale, "v_scale", torch.float32, 1, dev)
    args = _pack_rope(pq, pk, pv, ld_q, ld_k, ld_v, T, Hq, Hkv, D, rot, 1 if interleaved else 0,
                      eps, pp, pc, max_pos, qw, kw, po, ld_o, qs, ps, pkc, pvc, ks, vs, pages,
                      page, page_stride, slot_stride, head_stride)
    _check(_block_lib().fp8rl_rope_kv_append(args, _raw_stream(dev)), "fp8rl_rope_kv_append")
    return q_out
