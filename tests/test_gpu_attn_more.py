"""GPU parity of attention where work is found by the longer way: more documents than a wave has lanes,
of several tiles each, and sequences that were cut into more parts than a wave joins at a time. Bounds
are those of the tests whose helpers these are."""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from tests.gpu_util import assert_within
from tests.test_gpu_attn_decode import check, f64
from tests.test_gpu_attn_docs import Docs, check_bwd, check_fwd, i32

pytestmark = pytest.mark.gpu

# around one, two and three tiles of 128 rows, empty documents between them
SOME = [0, 1, 127, 128, 129, 3, 260, 0, 64, 257, 2, 0, 31, 256]


def many(docs):
    return [SOME[(5 * i) % len(SOME)] if i % 3 else i % 7 for i in range(docs)]


@pytest.mark.parametrize("heads", [(2, 1), (16, 8)])  # a key's queries in parts, and not
@pytest.mark.parametrize("more", [{}, dict(causal=False), dict(window=100, prefix=True),
                                  dict(cap=5.0, slopes=True, window=140)])
def test_more_documents_than_lanes(more, heads):
    nq = many(65 if heads[0] == 2 else 80)
    more = dict(more)
    if more.get("prefix"):
        more["prefix"] = [(37 * i) % 150 for i in range(len(nq))]
    d = Docs(nq, Hq=heads[0], Hkv=heads[1], D=64 if heads[0] == 2 else 16, seed=len(nq), **more)
    check_fwd(d)
    check_bwd(d)


@pytest.mark.parametrize("more", [{}, dict(causal=False, window=60), dict(window=90, prefix=True)])
def test_more_documents_than_lanes_of_other_lengths_than_their_keys(more):
    """Chunks behind cached keys, and some with fewer keys than queries."""
    nq = many(72)
    nk = [max(0, n + (0, 130, -40, 7, 300, -200)[i % 6]) for i, n in enumerate(nq)]
    more = dict(more)
    if more.get("prefix"):
        more["prefix"] = [(53 * i) % 200 for i in range(len(nq))]
    d = Docs(nq, nk, Hq=2, Hkv=1, D=128, seed=2, **more)
    check_fwd(d)
    check_bwd(d)


@pytest.mark.parametrize("docs", [63, 64, 65])
def test_as_many_documents_as_lanes(docs):
    d = Docs(many(docs), Hq=2, Hkv=2, D=64, seed=docs)
    check_fwd(d)
    check_bwd(d)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("Hkv,short,long", [(1, [40, 0, 3] * 50, 4100), (8, [33] * 20, 3000)])
def test_a_long_sequence_among_many(Hkv, short, long, codes):
    """More than sixteen parts of a sequence for one wave to join (units of 32 keys, two at least a
    part, 2048 / heads parts in all, one wave to a sequence and head up to sixteen parts on the
    average)."""
    lens = short[:7] + [long] + short[7:]
    units = np.array([-(-n // 32) for n in lens])
    lots = 2048 // Hkv
    per = max(2, -(-units.sum() // lots))
    assert lots <= 16 * len(lens) and -(-long // 32) / per > 17
    check(lens, 2 * Hkv, Hkv, 64, codes=codes, seed=Hkv)


@pytest.mark.parametrize("D", [16, 144])
def test_as_many_workgroups_as_a_launch_takes(D):
    """Documents of a few rows behind half a million without any: one workgroup of 512 threads less
    than makes 2^32. With one document more the call is refused, and nothing written."""
    some = Docs([5, 130], Hq=16, Hkv=16, D=D, seed=4)
    # (rows / 128 + documents) * heads = 2^23 less one workgroup for each head
    empty = [int(some.oq[0])] * ((1 << 19) - 1 - some.Tq // 128 - len(some.nq))
    most, past = i32(empty + some.oq.tolist()), i32(empty + empty[:1] + some.oq.tolist())
    args = dict(some.args, k_offsets=most)
    out, lse = fq.attn_fwd(*some.dev, D, most, **args)
    (want, tol), (wlse, ltol) = some.solve()
    rows = slice(some.oq[0], some.oq[-1])
    assert_within(f64(out)[rows], want[rows], tol[rows], "out")
    assert_within(f64(lse)[:, rows], wlse[:, rows], ltol[:, rows], "lse")
    sevens = [torch.full_like(t, 7.0) for t in some.dev]
    if D > 128:  # (no gradients)
        with pytest.raises(fq.Fp8rlError):
            fq.attn_fwd(*some.dev, D, past, **dict(args, k_offsets=past), out=sevens[0])
    else:
        dout = some.dout.cuda()
        grads = fq.attn_bwd(dout, *some.dev, out, lse, D, most, **args)
        # the same without the empty documents: a key's queries in parts, and so other sums
        same = fq.attn_bwd(dout, *some.dev, out, lse, D, some.q_offsets, **some.args)
        for a, b in zip(grads, same):
            assert (a[rows] - b[rows]).abs().max() <= 2.0 ** -7 * b[rows].abs().max()
        with pytest.raises(fq.Fp8rlError):
            fq.attn_bwd(dout, *some.dev, out, lse, D, past, **dict(args, k_offsets=past), dq=sevens[0],
                        dk=sevens[1], dv=sevens[2])
    assert all((t == 7).all() for t in sevens)
