"""The operators between the FP8 linears, in float64. TEST INFRASTRUCTURE.

Plain statements of the definitions in include/fp8rl_block.h, on float64 arrays that hold the bf16
or float32 input values exactly:

* B1: the stream h = bf16(x + residual) is rounded once (the float32 sum of two bf16 values and its
  rounding to bf16 give the same bits as one rounding of the exact sum: where the float32 sum is
  inexact, the smaller term lies below 2^-16 of the larger and cannot put the sum near a bf16
  midpoint), and the norm is taken of the stored h;
* B2: codes of y / S are those of 448 p / max|p| with p = h * weight, since the row's statistic
  cancels; S = max|y| / 448, 1 where max|y| == 0;
* B3: grouped rows are ordered by expert, then by (token, choice).
"""

from __future__ import annotations

import numpy as np

from . import e4m3
from .gemm import bf16_bits_to_f64, round_f64_to_bf16_bits


def to_bf16(v) -> np.ndarray:
    """float64 values rounded to bf16 and back."""
    return bf16_bits_to_f64(round_f64_to_bf16_bits(v))


def add_rmsnorm(x, residual, weight, eps):
    """(h, y): B1, in float64."""
    h = x if residual is None else to_bf16(x + residual)
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h, h * weight * r


def quant_rows(h, weight, y):
    """B2 with float32-type scales: (codes uint8 [M][K], S float64 [M][K/128])."""
    M, K = h.shape
    p = (h * weight).reshape(M, K // 128, 128)
    top = np.abs(p).max(axis=2, keepdims=True)
    q = np.where(top == 0, p, 448.0 * p / np.where(top == 0, 1.0, top))
    S = np.abs(y).reshape(M, K // 128, 128).max(axis=2) / 448.0
    return e4m3.encode(q.astype(np.float32)).reshape(M, K), np.where(S == 0, 1.0, S)


def add_rmsnorm_bwd(dy, h, weight, dh, eps):
    """(dx, dw, size of dx's terms, size of dw's terms): the sizes are the sums of magnitudes that
    the rounding errors of a float32 evaluation scale with."""
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    g = dy * weight
    dx = r * (g - h * r * r * np.mean(g * h, axis=1, keepdims=True))
    size = r * (np.abs(g) + np.abs(h) * r * r * np.mean(np.abs(g * h), axis=1, keepdims=True))
    if dh is not None:
        dx, size = dx + dh, size + np.abs(dh)
    t = dy * h * r
    return dx, t.sum(axis=0), size, np.abs(t).sum(axis=0)


def moe_sort(ids, E):
    """B3: (expert_offsets [E+1], row_ids [T*k], pos [T][k]) by walking the choices."""
    ids = np.asarray(ids)
    T, k = ids.shape
    lists = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < E:
                lists[e].append((t, j))
    offsets = np.zeros(E + 1, np.int32)
    row_ids = np.full(T * k, -1, np.int32)
    pos = np.full((T, k), -1, np.int32)
    row = 0
    for e in range(E):
        for t, j in lists[e]:
            row_ids[row], pos[t, j] = t, row
            row += 1
        offsets[e + 1] = row
    return offsets, row_ids, pos


def moe_combine(y, pos, weights):
    """(out, sum of magnitudes) in float64; choices outside [0, R) add nothing."""
    T, k = pos.shape
    out = np.zeros((T, y.shape[1]))
    size = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < y.shape[0]:
                term = (1.0 if weights is None else float(weights[t, j])) * y[pos[t, j]]
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def moe_dweights(dout, y, pos):
    """(dweights, sum of magnitudes) in float64."""
    T, k = pos.shape
    d, size = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < y.shape[0]:
                term = dout[t] * y[pos[t, j]]
                d[t, j], size[t, j] = term.sum(), np.abs(term).sum()
    return d, size


def rope(x, weight, eps, cos, sin, rot, interleaved):
    """One head per row, x [n][D], cos and sin [n][rot/2]: (rotated rows, size of the terms)."""
    u = x
    if weight is not None:
        u = x * weight / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)
    half = rot // 2
    a = 2 * np.arange(half) if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    out, size = u.copy(), np.abs(u)
    out[:, a] = u[:, a] * cos - u[:, b] * sin
    out[:, b] = u[:, b] * cos + u[:, a] * sin
    size[:, a] = np.abs(u[:, a] * cos) + np.abs(u[:, b] * sin)
    size[:, b] = np.abs(u[:, b] * cos) + np.abs(u[:, a] * sin)
    return out, size
