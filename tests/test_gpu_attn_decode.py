"""GPU parity of attention over the paged cache, and of the cache read back, against oracle.attn.

How far out may be off, with U = 2^-24 (half a step of float32) and one row's terms:
* a score is a sum of D products, exact in float32, then scaled (at most 4 roundings), capped (tanh by
  an exponential and a reciprocal, each within a few steps of float32: 8 U of the cap in all) and
  shifted by the slopes' term (3 roundings):
  da = D U size + 8 U (|a| + cap) + 3 U slope L, plus U |a| for the exponent's argument in each of the
  weight and the reference: 2 U (|a| + |top|);
* a weight is off by 2 da of itself (its own score and those in the sum), 4 U for two exponentials,
  and by its rounding for the product with v: 2^-11 of itself with an E4M3 cache (fp16; 2^-25 at least, of
  the largest weight), 2^-16 with a bf16 one (two bf16 terms, 2^-8 of 2^-8);
* sums of L terms are off by L U of the terms' magnitudes, twice (the numerator and the sum of the
  weights), the parts' factors and joins by 8 U;
* out is rounded once, 2^-8 of its value.
"""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from oracle import attn as oa
from oracle import e4m3
from tests.gpu_util import assert_within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
NAN = float("nan")


def f64(t):
    return t.detach().double().cpu().numpy()


def one(x):
    return torch.tensor([x], dtype=torch.float32, device="cuda")


class Paged:
    """Caches of N(0, 1) rows for sequences of these lengths, pages in random order, NaN in every
    place that no sequence has; table entries behind a sequence's last page are garbage. The table
    has room for `wide` keys at least (a call with a wide table splits short sequences too)."""

    def __init__(self, lens, Hkv, D, *, page=16, codes=True, heads_first=False, seed=0, spare=2,
                 wide=0):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.D, self.page, self.codes = lens, Hkv, D, page, codes
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        width = max(need + [1, -(-wide // page)]) + 1
        self.table = rng.integers(-5, 2 ** 31 - 1, (len(lens), width)).astype(np.int32)
        self.table[rng.random(self.table.shape) < 0.5] = -1
        shape = (pages, Hkv, page, D) if heads_first else (pages, page, Hkv, D)
        self.scale = {"k": 0.0171, "v": 0.0093} if codes else {"k": 1.0, "v": 1.0}
        self.raw, self.val = {}, {}
        for x in "kv":
            dense = rng.standard_normal((pages, page, Hkv, D))
            if codes:
                t = torch.from_numpy(dense / self.scale[x]).float().clamp(-448, 448)
                t = t.to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                t = torch.from_numpy(dense).to(torch.bfloat16)
            live = torch.zeros(pages, page, dtype=torch.bool)
            at = 0
            for b, n in enumerate(lens):
                mine = order[at:at + need[b]]
                at += need[b]
                self.table[b, :need[b]] = mine
                for i, pg in enumerate(mine):
                    live[pg, :min(page, n - i * page)] = True
            t[~live] = 0x7F if codes else NAN
            val = e4m3.decode(t.numpy()) * np.float64(np.float32(self.scale[x])) if codes else f64(t)
            self.val[x] = val
            dev = torch.empty(shape, dtype=t.dtype, device="cuda")
            view = dev.transpose(1, 2) if heads_first else dev
            view.copy_(t.cuda())
            self.raw[x] = view
        self.dev_table = torch.from_numpy(self.table).cuda()
        self.dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.scales = dict(k_scale=one(self.scale["k"]), v_scale=one(self.scale["v"])) if codes else {}

    def rows(self, x, b, n):
        """(values [n][Hkv][D], which of them exist)."""
        got = [oa.cached_row(self.val[x], self.table[b], j) for j in range(n)]
        there = np.array([r is not None for r in got], dtype=bool)
        zero = np.zeros((self.Hkv, self.D))
        return np.array([zero if r is None else r for r in got]).reshape(n, self.Hkv, self.D), there


def queries(B, Hq, D, q8, seed):
    t = torch.randn((B, Hq * D), generator=torch.Generator().manual_seed(seed))
    if q8:
        codes = (t / 0.0137).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return codes.cuda(), e4m3.decode(codes.numpy()) * np.float64(np.float32(0.0137))
    t = t.to(torch.bfloat16)
    return t.cuda(), f64(t)


def expected(paged, q, Hq, lens, *, sm_scale, window=0, cap=0.0, slopes=None):
    """(out, how far off it may be) [B][Hq * D]."""
    B, D, G = len(lens), paged.D, Hq // paged.Hkv
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        (k, there), (v, _) = paged.rows("k", b, n), paged.rows("v", b, n)
        first = max(0, n - window) if window else 0
        j = np.arange(n)[first:][there[first:]]
        if not len(j):
            continue
        for h in range(Hq):
            kh, vh = k[j, h // G], v[j, h // G]
            slope = 0.0 if slopes is None else float(slopes[h])
            o, _, w, ok, size, a = oa.attend(q[b].reshape(Hq, D)[h:h + 1], kh, vh, [n - 1], j,
                                             sm_scale=sm_scale, window=window, cap=cap, slope=slope)
            assert ok.all()
            big = np.abs(a).max()
            da = D * U * size.max() + 8 * U * (big + cap) + 3 * U * slope * n + 4 * U * big
            rel = 2 * da + 4 * U + (2.0 ** -11 if paged.codes else 2.0 ** -16) + 2 * len(j) * U + 8 * U
            small = 2.0 ** -25 * w.max() * np.abs(vh).sum(0) if paged.codes else 0.0
            out[b, h] = o[0]
            tol[b, h] = BF * np.abs(o[0]) + rel * (w[0] @ np.abs(vh)) + small
    return out.reshape(B, -1), tol.reshape(B, -1)


def check(lens, Hq, Hkv, D, *, q8=False, window=0, cap=0.0, slopes=False, sm_scale=None, seed=0,
          **cache):
    paged = Paged(lens, Hkv, D, seed=seed, **cache)
    B = len(lens)
    q, qv = queries(B, Hq, D, q8, seed + 1)
    sl = (2.0 ** -(8 * (torch.arange(Hq) + 1) / Hq)).float() if slopes else None
    out = fq.attn_decode(q, paged.raw["k"], paged.raw["v"], paged.dev_table, paged.dev_lens,
                         sm_scale=sm_scale, window=window, cap=cap,
                         slopes=None if sl is None else sl.cuda(), q_scale=one(0.0137) if q8 else None,
                         **paged.scales)
    want, tol = expected(paged, qv, Hq, lens, sm_scale=D ** -0.5 if sm_scale is None else sm_scale,
                         window=window, cap=cap, slopes=sl)
    assert_within(f64(out), want, tol + 1e-30, f"decode {lens[:4]} {Hq}/{Hkv}x{D}")
    return out


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("lens", [[1], [0], [31, 32, 33], [0, 1, 127, 128, 129, 0], [513, 2, 1100]])
def test_lengths(lens, codes):
    check(lens, 8, 2, 128, codes=codes, q8=codes)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 128, 144, 192, 256])
def test_head_widths(D, codes):
    check([77, 300], 6, 2, D, codes=codes, q8=not codes, seed=D)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (7, 1), (16, 1), (17, 1), (40, 2), (64, 4)])
def test_groups(Hq, Hkv):
    check([65, 700], Hq, Hkv, 64, codes=Hq % 2 == 0, seed=Hq)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("heads_first", [True, False])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 1024])
def test_pages(page, heads_first, codes):
    check([250, 61, 800], 4, 2, 64, page=page, heads_first=heads_first, codes=codes, seed=page)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("more", [dict(window=1), dict(window=100), dict(window=5000), dict(cap=2.5),
                                  dict(cap=50.0, window=300), dict(slopes=True),
                                  dict(slopes=True, cap=8.0, window=700), dict(sm_scale=3.0),
                                  dict(sm_scale=-0.5), dict(sm_scale=0.0)])
def test_scores_and_masks(more, codes):
    check([1, 99, 1400], 8, 4, 128, codes=codes, seed=7, **more)


@pytest.mark.parametrize("codes", [True, False])
def test_split_sequences(codes):
    """Uneven sequences in many pieces each, one of them alone in its call too."""
    check([9000], 4, 1, 64, codes=codes, seed=5)
    check([5000, 3, 0, 2049, 640, 12001], 4, 2, 64, codes=codes, seed=6)
    check([7001, 6000], 4, 2, 64, codes=codes, seed=8, window=2500)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 128, 144, 192, 256])
def test_split_head_widths(D, codes):
    check([77, 300, 0, 64], 6, 2, D, codes=codes, q8=not codes, seed=D, wide=4096)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("heads_first", [True, False])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 1024])
def test_split_pages(page, heads_first, codes):
    check([250, 61, 400], 4, 2, 64, page=page, heads_first=heads_first, codes=codes, seed=page,
          wide=2048)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (16, 1), (17, 1), (40, 2), (64, 4)])
def test_split_groups(Hq, Hkv):
    check([65, 300], Hq, Hkv, 64, codes=Hq % 2 == 0, seed=Hq, wide=2000)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("room", [400, 511, 512, 800, 1023, 1024])
def test_room_around_the_split(room, D, codes):
    """Tables with room for about as many keys as are not split (one more than the longest has)."""
    check([room, 5, room - 30], 2, 1, D, codes=codes, page=1, seed=room)


def test_many_sequences():
    rng = np.random.default_rng(2)
    check(rng.integers(0, 90, 300).tolist(), 4, 2, 32, codes=True, seed=9)
    check(rng.integers(0, 1500, 70).tolist(), 2, 2, 16, codes=False, seed=10)


def test_many_sequences_of_a_wide_table():
    rng = np.random.default_rng(3)
    check(rng.integers(0, 90, 300).tolist(), 4, 2, 32, codes=True, seed=9, wide=2000)
    check([0] * 130 + [400] + [0] * 80 + [65, 1], 2, 1, 16, codes=False, seed=9, wide=2000)


def test_bad_pages_are_not_seen():
    paged = Paged([600, 40], 2, 64, seed=3)
    paged.table[0, 3] = -1
    paged.table[0, 20] = 2 ** 30
    paged.table[0, 30] = paged.val["k"].shape[0]
    paged.table[1, :] = -7
    q, qv = queries(2, 4, 64, False, 4)
    out = fq.attn_decode(q, paged.raw["k"], paged.raw["v"], torch.from_numpy(paged.table).cuda(),
                         paged.dev_lens, **paged.scales)
    want, tol = expected(paged, qv, 4, [600, 40], sm_scale=1 / 8)
    assert_within(f64(out), want, tol + 1e-30, "bad pages")
    assert (want[1] == 0).all() and (out[1] == 0).all()


def test_lengths_outside_the_table_and_no_pages():
    paged = Paged([64, 64], 1, 32, seed=3, page=16)
    table = paged.dev_table[:, :4].contiguous()
    q, qv = queries(2, 2, 32, False, 4)
    args = (q, paged.raw["k"], paged.raw["v"])
    out = fq.attn_decode(*args, table, torch.tensor([2 ** 31 - 1, -4], dtype=torch.int32,
                                                    device="cuda"), **paged.scales)
    want, tol = expected(paged, qv, 2, [64, -4], sm_scale=32 ** -0.5)
    assert_within(f64(out), want, tol + 1e-30, "clamped")
    out = fq.attn_decode(*args, table[:, :0], paged.dev_lens, **paged.scales)
    assert (out == 0).all()
    none = paged.raw["k"][:0]
    out = fq.attn_decode(q, none, none, table, paged.dev_lens, **paged.scales)
    assert (out == 0).all()
    assert fq.attn_decode(q[:0], *args[1:], table[:0], paged.dev_lens[:0], **paged.scales).shape == (0, 64)


def test_a_nan_that_is_seen_shows():
    paged = Paged([40, 40], 1, 64, codes=False, seed=3)
    q, _ = queries(2, 2, 64, False, 4)
    q[0, :64] = NAN
    page, place = int(paged.table[1, 1]), 3
    paged.raw["v"][page, place, 0, 5] = float("inf")
    out = fq.attn_decode(q, paged.raw["k"], paged.raw["v"], paged.dev_table, paged.dev_lens)
    assert out[0, :64].isnan().all() and out[0, 64:].isfinite().all()
    bad = torch.zeros(128, dtype=torch.bool)
    bad[[5, 69]] = True
    assert torch.equal(~out[1].isfinite().cpu(), bad)


@pytest.mark.parametrize("codes", [True, False])
def test_rows_past_32_bit_offsets(codes):
    """Pages more than 2^32 bytes apart."""
    kind = torch.uint8 if codes else torch.bfloat16
    far = (1 << 32) + 4096 if codes else (1 << 31) + 4096
    paged = Paged([60], 2, 64, page=32, codes=codes, seed=12, spare=0)
    caches = []
    for x in "kv":
        flat = torch.empty(far + 32 * 2 * 64, dtype=kind, device="cuda")
        view = flat.as_strided((2, 32, 2, 64), (far, 128, 64, 1))
        view.copy_(paged.raw[x])
        caches.append(view)
    q, qv = queries(1, 4, 64, False, 4)
    out = fq.attn_decode(q, *caches, paged.dev_table, paged.dev_lens, **paged.scales)
    want, tol = expected(paged, qv, 4, [60], sm_scale=1 / 8)
    assert_within(f64(out), want, tol + 1e-30, "far pages")
    offsets = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    k, v = fq.kv_read(*caches, paged.dev_table, offsets, rows=60, **paged.scales)
    assert_read(paged, k, 0, 0, 60, "k")
    assert_read(paged, v, 0, 0, 60, "v")


def test_pitched_rows_and_unaligned_codes():
    """q and out as column slices; an E4M3 cache whose rows begin at odd multiples of 8 bytes."""
    paged = Paged([70, 33], 2, 80, seed=1)
    caches = []
    for x in "kv":
        raw = paged.raw[x]
        wide = torch.zeros((raw.shape[0], 16, 2, 88), dtype=torch.uint8, device="cuda")
        view = wide[..., 8:]
        view.copy_(raw)
        caches.append(view)
    q, qv = queries(2, 4, 80, False, 2)
    buf = torch.full((2, 1000), 3.0, dtype=torch.bfloat16, device="cuda")
    buf[:, 8:328] = q
    fq.attn_decode(buf[:, 8:328], *caches, paged.dev_table, paged.dev_lens, out=buf[:, 400:720],
                   **paged.scales)
    want, tol = expected(paged, qv, 4, [70, 33], sm_scale=80 ** -0.5)
    assert_within(f64(buf[:, 400:720]), want, tol + 1e-30, "pitched")
    rest = torch.cat([buf[:, :8], buf[:, 328:400], buf[:, 720:]], dim=1)
    assert (rest == 3).all()


def test_repeats_and_workspace_contents():
    """The same bits again, whatever the workspace held."""
    paged = Paged([3000, 700], 2, 64, seed=1)
    q, _ = queries(2, 4, 64, False, 2)
    need = fq.fp8rl_attn_decode_workspace_bytes(2, 4, 2, 64, paged.table.shape[1] * 16)
    assert need > 0
    got = []
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got.append(fq.attn_decode(q, paged.raw["k"], paged.raw["v"], paged.dev_table, paged.dev_lens,
                                  workspace=ws, **paged.scales))
    got.append(fq.attn_decode(q, paged.raw["k"], paged.raw["v"], paged.dev_table, paged.dev_lens,
                              **paged.scales))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    with pytest.raises(fq.Fp8rlError):
        fq.attn_decode(q, paged.raw["k"], paged.raw["v"], paged.dev_table, paged.dev_lens,
                       workspace=ws[:need - 1], **paged.scales)


# ------------------------------------------------------------------------------ the cache read back


def assert_read(paged, got, b, first, n, x):
    """Rows of sequence b from key `first` on: E4M3 code * scale in float32, rounded to bf16."""
    want, there = paged.rows(x, b, first + n)
    assert there.all()
    if paged.codes:
        raw = want / np.float64(np.float32(paged.scale[x]))
        want = raw.astype(np.float32) * np.float32(paged.scale[x])
    want = torch.from_numpy(want[first:].reshape(n, paged.Hkv * paged.D)).to(torch.bfloat16)
    assert torch.equal(got.cpu(), want), (x, b)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("D,Hkv,page,heads_first", [(128, 8, 16, False), (64, 2, 24, True),
                                                    (8, 1, 1, False), (80, 3, 7, True),
                                                    (512, 2, 64, False)])
def test_read(D, Hkv, page, heads_first, codes):
    starts, lens = [0, 5, 0, 33, 0], [1, 70, 0, 3, 130]
    paged = Paged([a + b for a, b in zip(starts, lens)], Hkv, D, page=page, codes=codes,
                  heads_first=heads_first, seed=D)
    off = np.concatenate([[2], 2 + np.cumsum(lens)])
    R = int(off[-1]) + 9
    k = torch.full((R, Hkv * D + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full((R, Hkv * D), 5.0, dtype=torch.bfloat16, device="cuda")
    got = fq.kv_read(paged.raw["k"], paged.raw["v"], paged.dev_table,
                     torch.from_numpy(off.astype(np.int32)).cuda(),
                     starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), k_out=k[:, :-8],
                     v_out=v, **paged.scales)
    assert got[1] is v
    for b, n in enumerate(lens):
        at = slice(int(off[b]), int(off[b + 1]))
        assert_read(paged, k[at, :-8], b, starts[b], n, "k")
        assert_read(paged, v[at], b, starts[b], n, "v")
    assert (k[:2] == 5).all() and (k[off[-1]:] == 5).all() and (k[:, -8:] == 5).all()
    assert (v[:2] == 5).all() and (v[off[-1]:] == 5).all()


def test_read_many_sequences():
    """More sequences than one search step covers, empty ones in rows of hundreds."""
    rng = np.random.default_rng(0)
    lens = np.where(rng.random(5000) < 0.9, 0, rng.integers(1, 4, 5000))
    paged = Paged(lens.tolist(), 1, 8, page=2, seed=1)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = fq.kv_read(paged.raw["k"], paged.raw["v"], paged.dev_table, torch.from_numpy(off).cuda(),
                      rows=int(off[-1]), **paged.scales)
    for b in np.nonzero(lens)[0]:
        assert_read(paged, k[off[b]:off[b + 1]], b, 0, int(lens[b]), "k")
        assert_read(paged, v[off[b]:off[b + 1]], b, 0, int(lens[b]), "v")


def test_read_of_what_is_not_there_writes_nothing():
    paged = Paged([64, 64], 1, 8, page=16, seed=2)
    paged.table[0, 1] = -1
    paged.table[1, 2] = 10 ** 6
    k = torch.full((200, 8), 5.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    off = torch.tensor([0, 60, 200], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, -20], dtype=torch.int32, device="cuda")
    fq.kv_read(paged.raw["k"], paged.raw["v"], torch.from_numpy(paged.table[:, :4]).contiguous().cuda(),
               off, starts=starts, k_out=k, v_out=v, **paged.scales)
    live = np.zeros(200, dtype=bool)
    live[:16] = live[32:60] = True
    live[80:112] = live[128:144] = True  # keys 0 .. 31 and 48 .. 63 of the second
    untouched = torch.from_numpy(~live).cuda()
    for t in (k, v):
        assert (t[untouched] == 5).all() and not (t[~untouched] == 5).all(dim=1).any()
    before = k.clone()
    fq.kv_read(paged.raw["k"][:0], paged.raw["v"][:0], paged.dev_table, off, k_out=k, v_out=v,
               **paged.scales)
    assert torch.equal(k, before)
