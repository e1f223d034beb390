"""Attention whose result is made of small weights: one key takes the maximum with a value of zero, and
thousands of others, far below it, are what is left (float64, oracle.attn).

How far out may be off, with U = 2^-24 (half a step of float32) and the terms of one row:
* a score is a sum of D products, exact in float32, scaled, and off by da = D U size + 12 U |a| with the
  exponent's argument in the weight and the reference;
* a weight is off by 2 da of itself (its own score and those in the sum), by 4 U for two exponentials, and
  by its rounding for the product with v: 2^-16 of itself (two bf16 terms, 2^-8 of 2^-8), however small
  it is;
* sums of n terms are off by n U of the terms' magnitudes, numerator and denominator, joins by 8 U;
* out is rounded once, 2^-8 of its value.
"""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from oracle import attn as oa
from oracle import e4m3
from tests.gpu_util import assert_within
from tests.test_gpu_attn_docs import Docs, check_fwd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
D, PAGE = 64, 16


def f64(t):
    return t.detach().double().cpu().numpy()


def stored(values, scale):
    """(as a cache holds it, what it stands for in float64): E4M3 codes with a scale, bf16 without."""
    t = torch.from_numpy(values)
    if scale is None:
        t = t.to(torch.bfloat16)
        return t, f64(t)
    t = (t / scale).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return t, e4m3.decode(t.numpy()) * np.float64(np.float32(scale))


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("n", [700, 9000])  # a workgroup's, and one that is split
@pytest.mark.parametrize("gap", [8, 12, 17, 18, 25, 60])
def test_decode_of_a_tail_behind_a_key_without_value(gap, n, codes):
    """Scores of the tail are N(0, 1), the first (of the second sequence the last) key's is `gap`."""
    rng = np.random.default_rng(gap)
    pages = -(-n // PAGE)
    table = torch.arange(2 * pages, dtype=torch.int32, device="cuda").view(2, pages)
    sinks = (0, n - 1)
    cache, rows = {}, {}
    for x, scale in (("k", gap / 256), ("v", 0.0117)):
        dense = np.zeros((2, pages * PAGE, D))
        dense[:, :n] = rng.standard_normal((2, n, D)) + (x == "v")
        for b, at in enumerate(sinks):
            dense[b, at] = 0
        if x == "k":
            dense[:, :, 0] = 0
            for b, at in enumerate(sinks):
                dense[b, at, 0] = gap
        raw, val = stored(dense, scale if codes else None)
        cache[x] = raw.view(2 * pages, PAGE, 1, D).cuda()
        rows[x] = val[:, :n]
    q = torch.from_numpy(rng.standard_normal((2, D)) / 8)
    q[:, 0] = 1
    q = q.to(torch.bfloat16)
    scales = dict(k_scale=torch.tensor([gap / 256], device="cuda"),
                  v_scale=torch.tensor([0.0117], device="cuda")) if codes else {}
    out = fq.attn_decode(q.cuda(), cache["k"], cache["v"], table,
                         torch.tensor([n, n], dtype=torch.int32, device="cuda"), sm_scale=1.0, **scales)
    want, tol = np.zeros((2, D)), np.zeros((2, D))
    for b in range(2):
        o, _, w, _, size, a = oa.attend(f64(q[b:b + 1]), rows["k"][b], rows["v"][b], [n - 1],
                                        np.arange(n), sm_scale=1.0)
        da = D * U * size.max() + 12 * U * np.abs(a).max()
        rel = 2 * da + 4 * U + 2.0 ** -16 + 2 * n * U + 8 * U
        want[b], tol[b] = o[0], BF * np.abs(o[0]) + rel * (w[0] @ np.abs(rows["v"][b]))
    assert_within(f64(out), want, tol, f"tail {gap} below, {n} keys")


@pytest.mark.parametrize("gap", [17, 40])
def test_documents_behind_a_key_without_value(gap):
    d = Docs([300, 140], D=64, Hq=2, Hkv=1, seed=3, sm_scale=1.0)
    d.q *= 0.125
    d.q[:, ::64] = 1
    d.k[:, 0] = 0
    for first in d.oq[:-1]:
        d.k[first] = 0
        d.k[first, 0] = gap
        d.v[first] = 0
    d.dev = d.q.cuda(), d.k.cuda(), d.v.cuda()
    check_fwd(d)
