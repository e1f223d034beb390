"""The largest sizes that include/fp8rl_attn.h admits, from both sides (CPU only: no kernel is ever
launched here). A dispatch has fewer than 2^32 threads, and some kernels have 512 to a workgroup."""

import ctypes

import pytest

from fp8_blockwise_quantization_amd import _attn
from tests.test_abi_attn_host import A, CACHE, DOCS, ENULL, ESHAPE, EWS, L  # noqa: F401  (L: the fixture)


def docs_args(**k):
    a = dict(DOCS, **k)
    qc, kc = a["q_heads"] * a["head_dim"], a["kv_heads"] * a["head_dim"]
    a.update({n: qc for n in ("ld_q", "ld_out", "ld_dout", "ld_dq")})
    a.update({n: kc for n in ("ld_k", "ld_v", "ld_dk", "ld_dv")})
    return _attn.AttnArgs(**a)


# sizes whose tiles of 128 rows and head counts come to one workgroup less than 2^23 or 2^24, or to it:
# documents, rows, heads
BELOW_23 = [((1 << 19) - 1, 100, 16), (1, (1 << 23) - 129, 128), (5, 100, 4)]
FROM_23 = [(1 << 19, 100, 16), (1, (1 << 23) - 128, 128), (100, 1 << 23, 4096)]
BELOW_24 = [((1 << 20) - 1, 100, 16), (1, (1 << 24) - 129, 128)]


@pytest.mark.parametrize("head_dim,few", [(16, True), (128, True), (144, False), (256, False)])
def test_forward(L, head_dim, few):  # noqa: F811
    def call(docs, T, heads):
        # (behind the sizes' check there is no q)
        a = docs_args(docs=docs, Tq=T, Tk=50, q_heads=heads, kv_heads=heads, head_dim=head_dim, q=None)
        return L.fp8rl_attn_fwd(ctypes.byref(a), None)

    for size in BELOW_23:
        assert call(*size) == ENULL, size
    for size in FROM_23[:2] + BELOW_24:
        assert call(*size) == (ENULL if few else ESHAPE), size
    assert call(*FROM_23[2]) == ESHAPE  # 2^28
    # the keys' rows do not count among its workgroups
    a = docs_args(docs=1, Tq=128, Tk=(1 << 24) - 1, q_heads=100, kv_heads=1, head_dim=head_dim, q=None)
    assert L.fp8rl_attn_fwd(ctypes.byref(a), None) == ENULL


def test_backward(L):  # noqa: F811
    need = L.fp8rl_attn_bwd_workspace_bytes

    def call(docs, Tq, Tk, heads, kv_heads):
        # (behind all other checks there is no workspace)
        a = docs_args(docs=docs, Tq=Tq, Tk=Tk, q_heads=heads, kv_heads=kv_heads, head_dim=16)
        got = L.fp8rl_attn_bwd(ctypes.byref(a), None, 0, None)
        assert (need(Tq, Tk, docs, heads, kv_heads, 16) > 0) == (got == EWS)
        return got

    for docs, T, heads in BELOW_23:
        assert call(docs, T, T, heads, heads) == EWS, (docs, T, heads)
        assert call(docs, 100, T, heads, heads) == EWS, (docs, T, heads)
    for docs, T, heads in FROM_23 + BELOW_24:
        assert call(docs, T, T, heads, heads) == ESHAPE, (docs, T, heads)
        assert call(docs, 100, T, heads, heads) == ESHAPE, (docs, T, heads)
    # a workgroup of the keys' has a key head
    for docs, T, heads in FROM_23[:2] + BELOW_24:
        assert call(docs, T, T, heads, heads // 2) == EWS, (docs, T, heads)
    # and the queries' rows do not count among these
    docs, T, heads = BELOW_24[1]
    assert call(docs, T, 100, heads, heads) == EWS


@pytest.mark.parametrize("page_size", [1, 3, 16])
def test_keys_of_all_sequences_of_a_decode(L, page_size):  # noqa: F811
    """B * table_width * page_size < 2^35, also where the page size does not divide that."""
    def call(B, width):
        a = _attn.AttnDecodeArgs(**dict(CACHE, page_size=page_size, page_stride=page_size * 256, q=A,
                                        ld_q=1024, B=B, q_heads=8, lengths=A, sm_scale=0.1, out=A,
                                        ld_out=1024, table_width=width, ld_table=width))
        return L.fp8rl_attn_decode(ctypes.byref(a), None, 0, None)

    pages = -(-(1 << 35) // page_size)  # of 2^35 keys, or just past them
    for B in (32, 43691, 65536):
        width = (pages - 1) // B
        if width * page_size <= 1 << 30:
            assert call(B, width) == EWS, (B, width)
        assert call(B, -(-pages // B)) == ESHAPE, (B, width)
