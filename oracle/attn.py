"""Attention of one document in float64: which keys a query sees, its scores, the weighted sum and its
gradients, and the paged cache's rows. Plain definitions, one query row against one key row at a
time where that is what the definition says.
"""

from __future__ import annotations

import numpy as np


def seen(p, j, *, causal=True, window=0, prefix=0):
    """[queries][keys]: whether the query at position p sees key j."""
    p, j = np.asarray(p)[:, None], np.asarray(j)[None, :]
    ok = np.ones((p.shape[0], j.shape[1]), dtype=bool)
    if causal:
        ok &= j <= p
    if window:
        ok &= p - j < window
    return ok | (j < prefix)


def scores(q, k, p, j, *, sm_scale, cap=0.0, slope=0.0):
    """(a, da/ds, size): the scores of all pairs, the cap's slope there, and sm_scale sum |q| |k|,
    the size of what a score is the sum of."""
    s = sm_scale * (q @ k.T)
    size = abs(sm_scale) * (np.abs(q) @ np.abs(k).T)
    t = np.tanh(s / cap) if cap else None
    a = cap * t if cap else s
    far = np.abs(np.asarray(p)[:, None] - np.asarray(j)[None, :])
    return a - slope * far, (1 - t * t if cap else np.ones_like(s)), size


def weights(a, ok):
    """(w, lse): softmax over the keys that are seen; a row that sees none has weights 0, lse -inf."""
    a = np.where(ok, a, -np.inf)
    top = a.max(axis=1, initial=-np.inf)
    ref = np.where(np.isfinite(top), top, 0.0)
    e = np.where(ok, np.exp(a - ref[:, None]), 0.0)
    total = e.sum(axis=1)
    some = ok.any(axis=1)
    with np.errstate(divide="ignore"):
        lse = np.where(some, np.log(total) + ref, -np.inf)
    return np.where(some[:, None], e / np.where(some, total, 1.0)[:, None], 0.0), lse


def attend(q, k, v, p, j, *, sm_scale, causal=True, window=0, prefix=0, cap=0.0, slope=0.0):
    """One head: (out, lse, weights, seen, sizes of the scores' terms, scores)."""
    ok = seen(p, j, causal=causal, window=window, prefix=prefix)
    a, _, size = scores(q, k, p, j, sm_scale=sm_scale, cap=cap, slope=slope)
    w, lse = weights(a, ok)
    return w @ np.where(ok.any(axis=0)[:, None], v, 0.0), lse, w, ok, size, a


def gradients(q, k, v, dout, p, j, *, sm_scale, causal=True, window=0, prefix=0, cap=0.0, slope=0.0):
    """One head: (dq, dk, dv) of <dout, out>, with the size of each (the same sums of magnitudes)."""
    ok = seen(p, j, causal=causal, window=window, prefix=prefix)
    a, slant, _ = scores(q, k, p, j, sm_scale=sm_scale, cap=cap, slope=slope)
    w, _ = weights(a, ok)
    dw = dout @ v.T
    mean = (w * dw).sum(axis=1, keepdims=True)
    ds = np.where(ok, sm_scale * w * (dw - mean) * slant, 0.0)
    # what ds is formed of: both terms' magnitudes, before they cancel and before the cap's slope
    big = w * ((np.abs(dout) @ np.abs(v).T) + (w @ np.abs(v) * np.abs(dout)).sum(1, keepdims=True))
    big = np.where(ok, abs(sm_scale) * big, 0.0)
    return ((ds @ k, ds.T @ q, w.T @ dout),
            (big @ np.abs(k), big.T @ np.abs(q), w.T @ np.abs(dout)))


def cached_row(cache, table_row, key):
    """Row `key` of one sequence, cache [page][place][head][D]; None where there is none."""
    pages, size = cache.shape[:2]
    i = key // size
    if key < 0 or i >= len(table_row) or not 0 <= table_row[i] < pages:
        return None
    return cache[table_row[i], key % size]
