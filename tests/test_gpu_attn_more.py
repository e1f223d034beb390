"""GPU parity of attention where work is found by the longer way: more documents than a wave has lanes,
of several tiles each, and sequences that were cut into more parts than a wave joins at a time. Bounds
are those of the tests whose helpers these are."""

import numpy as np
import pytest

from tests.test_gpu_attn_decode import check
from tests.test_gpu_attn_docs import Docs, check_bwd, check_fwd

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
