"""GPU parity of the rotated append to a paged cache against oracle.block and oracle.kvcache.

A rotated value is a product, a fused multiply-add (2 half steps, 2^-24, of the sum of the two
terms' magnitudes); a head norm before it adds a sum of at most 16 values in a lane and 5 steps
across lanes (half of 26 with the mean's roundings), the reciprocal square root and two products:
20 half steps in all. Rounding adds half a step of the result's type: bf16 2^-8 of the value, E4M3
2^-4 of it and at least 2^-10 (codes saturate at 448). v is neither normalised nor rotated: its
codes are those of the IEEE float32 quotient, bit for bit. Bytes that no token names stay.
"""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from oracle import block as ob
from oracle import e4m3
from oracle import kvcache as okv
from tests.gpu_util import assert_within, bits16
from workloads import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
FAR = 5000


def f64(t):
    return t.detach().double().cpu().numpy()


def table(rot, seed=1):
    i = np.arange(rot // 2)
    ang = np.arange(FAR)[:, None] * 1e4 ** (-2.0 * i / max(rot, 1))
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], axis=1)).float().cuda()


class Case:
    def __init__(self, T, Hq, Hkv, D, rot, *, pairs=False, norms=False, cache8=True, q8=False,
                 page=16, heads_first=False, seed=0, spare=3):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.__dict__.update(T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, pairs=pairs, cache8=cache8, q8=q8,
                             page=page)
        cols = (Hq + 2 * Hkv) * D
        fused = synth.act_bf16(max(T, 1), cols + 16, seed=seed)[:T].cuda()
        self.q = fused[:, :Hq * D] if Hq else None
        self.k = fused[:, Hq * D:(Hq + Hkv) * D]
        self.v = fused[:, (Hq + Hkv) * D:cols]
        w = lambda: (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()  # noqa: E731
        self.qw, self.kw = (w(), w()) if norms else (None, None)
        self.table = table(rot) if rot else None
        self.pos = torch.from_numpy(rng.integers(0, FAR, T)).cuda()
        pages = -(-T // page) + spare
        slots = rng.permutation(pages * page)[:T]
        slots[rng.random(T) < 0.1] = -1
        self.slots = torch.from_numpy(slots).cuda()
        shape = (pages, Hkv, page, D) if heads_first else (pages, page, Hkv, D)
        kind = torch.uint8 if cache8 else torch.bfloat16
        fill = lambda: (torch.from_numpy(rng.integers(0, 120, shape)).to(torch.uint8).cuda()  # noqa: E731
                        if cache8 else torch.from_numpy(rng.standard_normal(shape)).to(kind).cuda())
        raw = fill(), fill()
        self.kc, self.vc = (t.transpose(1, 2) if heads_first else t for t in raw)
        one = lambda x: torch.tensor([x], dtype=torch.float32, device="cuda")  # noqa: E731
        self.ks, self.vs = (one(0.0171), one(0.0093)) if cache8 else (None, None)
        self.qs = one(0.0137) if q8 else None

    def call(self, **more):
        a = dict(interleaved=self.pairs, q_weight=self.qw, k_weight=self.kw, q_scale=self.qs,
                 k_scale=self.ks, v_scale=self.vs)
        a.update(more)
        return fq.rope_kv_append(self.q, self.k, self.v, self.pos, self.table, self.slots, self.kc,
                                 self.vc, **a)

    def turned(self, x, weight):
        """Rotated rows [T][H][D] in float64 and the sizes of their terms."""
        H = x.shape[1] // self.D
        rows = f64(x).reshape(-1, self.D)
        half = self.rot // 2
        # (tokens outside the table are not compared)
        at = np.clip(self.pos.cpu().numpy(), 0, FAR - 1)
        cs = f64(self.table)[at] if self.rot else np.zeros((self.T, 0))
        cs = np.repeat(cs, H, axis=0)
        out, size = ob.rope(rows, None if weight is None else f64(weight), 1e-6, cs[:, :half],
                            cs[:, half:], self.rot, self.pairs)
        return out.reshape(self.T, H, self.D), size.reshape(self.T, H, self.D)


def check_values(got, want, size, scale, what):
    if scale is None:
        assert_within(f64(got), want, BF * np.abs(want) + 20 * U * size + 1e-40, what)
        return
    s = float(scale)
    v, slack = want / s, 20 * U * size / s
    bound = np.maximum(2.0 ** -4 * np.minimum(np.abs(v), 448), 2.0 ** -10) + slack
    assert_within(e4m3.decode(got.cpu().numpy()), np.clip(v, -448, 448), bound, what)


def check(c, skipped=()):
    before = c.kc.clone(), c.vc.clone()
    q0 = None if c.q is None else c.q.clone()
    out = c.call()
    torch.cuda.synchronize()
    slots = c.slots.cpu().numpy()
    live = np.array([0 <= s < c.kc.shape[0] * c.page and t not in skipped
                     for t, s in enumerate(slots)], dtype=bool)
    page, place = slots[live] // c.page, slots[live] % c.page
    if c.q is not None:
        want, size = c.turned(q0, c.qw)
        keep = [t for t in range(c.T) if t not in skipped]
        check_values(out.view(c.T, c.Hq, c.D)[keep], want[keep], size[keep], c.qs, "q")
    kw, ksize = c.turned(c.k, c.kw)
    check_values(c.kc[page, place], kw[live], ksize[live], c.ks, "k")
    v = c.v.reshape(c.T, c.Hkv, c.D)[live]
    if c.cache8:
        want = okv.quant_per_tensor(bits16(v), np.float32(float(c.vs)))
        assert np.array_equal(c.vc[page, place].cpu().numpy(), want)
    else:
        assert torch.equal(c.vc[page, place], v)
    rest = torch.ones(c.kc.shape[:2], dtype=torch.bool, device="cuda")
    rest[page, place] = False
    assert torch.equal(c.kc[rest], before[0][rest]) and torch.equal(c.vc[rest], before[1][rest])
    return out


@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [
    (1, 32, 8, 128, 128), (64, 32, 8, 128, 128), (3, 1, 1, 8, 0), (5, 2, 1, 16, 16),
    (33, 4, 2, 64, 64), (17, 6, 3, 80, 32), (9, 5, 1, 96, 96), (40, 7, 1, 72, 48),
    (12, 16, 2, 256, 128), (6, 3, 3, 512, 512), (21, 8, 4, 120, 112), (1000, 28, 4, 128, 128)])
def test_append_shapes(T, Hq, Hkv, D, rot, norms):
    print(f"[append] T={T} {Hq}/{Hkv} x {D} rot={rot} norms={norms}", flush=True)
    check(Case(T, Hq, Hkv, D, rot, norms=norms, seed=T + D))


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,more", [
    (9001, 24, 4, 16, 16, dict(norms=True)), (4500, 26, 3, 32, 16, dict(q8=True, pairs=True)),
    (2000, 32, 4, 64, 64, dict(heads_first=True, norms=True, q8=True)),
    (1003, 20, 4, 96, 96, dict(cache8=False)), (1000, 14, 2, 256, 128, dict(q8=True, norms=True)),
    (301, 24, 3, 512, 512, dict(cache8=False, pairs=True))])
def test_append_of_many_tokens(T, Hq, Hkv, D, rot, more):
    """Enough tokens for two heads a lane, at every number of lanes that share a head."""
    print(f"[append] T={T} {Hq}/{Hkv} x {D} rot={rot} {more}", flush=True)
    check(Case(T, Hq, Hkv, D, rot, seed=T, **more))


@pytest.mark.parametrize("cache8,q8", [(True, True), (True, False), (False, False), (False, True)])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_append_types_layouts_and_pages(cache8, q8, heads_first, pairs, page):
    print(f"[append] cache8={cache8} q8={q8} heads_first={heads_first} pairs={pairs} page={page}",
          flush=True)
    for D, rot in ((128, 128), (80, 48)):
        check(Case(50, 8, 2, D, rot, pairs=pairs, norms=True, cache8=cache8, q8=q8, page=page,
                   heads_first=heads_first, seed=page + D))


def test_append_without_q_and_padded_rows():
    check(Case(20, 0, 4, 128, 128, seed=3))
    c = Case(20, 8, 4, 128, 128, seed=4)
    c.slots[12:] = -1                               # rows behind the last sequence
    c.slots[3] = c.kc.shape[0] * c.page             # past the last page
    c.slots[4] = 2 ** 62
    c.slots[5] = -2 ** 63
    check(c)
    c = Case(20, 8, 4, 128, 128, seed=5)
    c.pos[2], c.pos[7] = -1, FAR                    # outside the table: skipped altogether
    q_out = torch.full((20, 8 * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    before = q_out.clone()
    kc, vc = c.kc.clone(), c.vc.clone()
    c.call(q_out=q_out)
    torch.cuda.synchronize()
    assert torch.equal(q_out[[2, 7]], before[[2, 7]])
    assert not torch.equal(q_out[3], before[3])
    for t in (2, 7):
        s = int(c.slots[t])
        if s >= 0:
            at = s // c.page, s % c.page
            assert torch.equal(c.kc[at], kc[at]) and torch.equal(c.vc[at], vc[at])
    check(c, skipped=(2, 7))


@pytest.mark.parametrize("norms", [False, True])
def test_codes_are_correctly_rounded(norms):
    """The codes of q and k are those of the float64 values: no value lands on the wrong side of a
    step (none of these lies within float64's error of one)."""
    c = Case(700, 8, 4, 128, 128, norms=norms, q8=True, seed=13, spare=9)
    c.slots = torch.arange(700, device="cuda")
    q = c.call()
    torch.cuda.synchronize()
    for got, x, w, s in ((q.view(700, 8, 128), c.q, c.qw, c.qs),
                         (c.kc.reshape(-1, 4, 128)[:700], c.k, c.kw, c.ks)):
        v = np.clip(c.turned(x, w)[0] / np.float64(float(s)), -448, 448)
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
        want = np.clip(np.rint(v / step) * step, -448, 448)
        # v is off by float64's roundings (and so may sit on the other side within 2^-45 of a tie)
        tie = np.abs(np.abs(v / step - np.floor(v / step)) - 0.5) < 2.0 ** -40
        assert np.array_equal(e4m3.decode(got.cpu().numpy())[~tie], want[~tie])


def test_append_q_in_place_equals_out_of_place():
    for norms in (False, True):
        c = Case(37, 8, 2, 128, 96, norms=norms, seed=6)
        want = c.call()
        c.q = c.q.clone()
        got = c.call(q_out=c.q)
        torch.cuda.synchronize()
        assert got.data_ptr() == c.q.data_ptr() and torch.equal(got, want)


def test_append_into_interleaved_keys_and_values():
    """One buffer [page][place][key or value][head][column]: two views with the same strides."""
    c = Case(30, 4, 2, 64, 64, seed=7)
    pages = c.kc.shape[0]
    both = torch.full((pages, c.page, 2, 2, 64), 0x11, dtype=torch.uint8, device="cuda")
    c.kc, c.vc = both[:, :, 0], both[:, :, 1]
    check(c)


def test_append_far_slots_pass_32_bits():
    """A cache whose last page lies beyond 2^32 bytes."""
    D, Hkv, page = 128, 8, 64
    pages = (1 << 32) // (page * Hkv * D) + 5
    c = Case(4, 2, Hkv, D, D, page=page, seed=8)
    big = torch.zeros((pages, page, Hkv, D), dtype=torch.uint8, device="cuda")
    c.kc = c.vc = big
    c.slots = torch.tensor([pages * page - 1, (pages - 3) * page + 1, 0, 77], device="cuda")
    c.kc = big
    c.vc = torch.zeros_like(big)
    c.call()
    torch.cuda.synchronize()
    want, size = c.turned(c.k, c.kw)
    s = c.slots
    check_values(c.kc[s // page, s % page], want, size, c.ks, "far k")
    v = okv.quant_per_tensor(bits16(c.v.reshape(4, Hkv, D)), np.float32(float(c.vs)))
    assert np.array_equal(c.vc[s // page, s % page].cpu().numpy(), v)
    # nothing else was written (reduced without a boolean copy of the 4 GiB)
    for cache in (c.kc, c.vc):
        cache[s // page, s % page] = 0
        assert int(cache.view(-1).view(torch.int64).abs().max()) == 0


def test_append_extreme_values_and_nan():
    c = Case(4, 1, 1, 32, 0, seed=9)
    c.slots = torch.tensor([0, 1, 2, 3], device="cuda")
    x = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    x[0, :4] = torch.tensor([3e38, -3e38, 1e-30, -1e-30])
    x[1, 0], x[1, 1], x[1, 2] = float("nan"), float("inf"), float("-inf")
    c.q, c.k, c.v = x, x, x
    c.call()
    torch.cuda.synchronize()
    for cache in (c.kc, c.vc):
        rows = cache[0, :4, 0].cpu().numpy()
        assert list(rows[0, :4]) == [0x7E, 0xFE, 0x00, 0x80]
        assert rows[1, 0] & 0x7F == 0x7F and list(rows[1, 1:3]) == [0x7E, 0xFE]
        assert not rows[2:].any()
    check(Case(0, 4, 2, 64, 64, seed=10, spare=1))


def test_append_equals_the_plain_store_without_rotation():
    """Nothing rotated, no norms: the same bytes as the slot-mapped per-tensor store."""
    c = Case(100, 0, 8, 128, 0, seed=11)
    flat = c.kc.clone().view(-1, 8 * 128)
    fq.quant_per_tensor(c.k, c.ks, flat, c.slots)
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.kc.view(-1, 8 * 128), flat)


def test_binding_refusals_on_device():
    c = Case(4, 2, 2, 64, 64, seed=12)
    with pytest.raises(ValueError):
        c.call(q_out=torch.empty((4, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        c.call(q_out=torch.empty((4, 128), dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        c.call(k_scale=None, v_scale=None)  # uint8 caches need scales
    with pytest.raises(fq.Fp8rlError):
        c.call(v_scale=None)
    c.vc = c.vc.transpose(1, 2).contiguous().transpose(1, 2)
    with pytest.raises(ValueError):
        c.call()
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fq.Fp8rlError):
        fq.add_rmsnorm_quant(x.expand(2, 128)[:1].expand(2, 128), w)  # rows of pitch 0
    with pytest.raises(ValueError):
        fq.add_rmsnorm_quant(x, w.cpu())
    with pytest.raises(ValueError):
        fq.add_rmsnorm_quant(x, w[:64])
    with pytest.raises(TypeError):
        fq.moe_sort(torch.zeros((2, 2), device="cuda"), 4)
    with pytest.raises(ValueError):
        fq.moe_sort(torch.zeros((2, 4), dtype=torch.int32, device="cuda")[:, ::2], 4)


@pytest.mark.parametrize("cache8,q8", [(True, True), (False, False)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T", [7, 2100])
def test_head_norms_of_far_values(T, pairs, cache8, q8):
    """Heads whose squares leave float32 are normalised like any other (the bounds are those of the
    module); a head with an infinity or a NaN is NaN throughout, and only that head."""
    print(f"[append] far heads T={T} pairs={pairs} cache8={cache8}", flush=True)
    H, D = 2, 128
    c = Case(T, H, H, D, 96, pairs=pairs, norms=True, cache8=cache8, q8=q8, seed=21)
    c.slots = torch.arange(T, device="cuda")
    g = torch.Generator().manual_seed(22)
    x = torch.randn((T, H, D), generator=g).clamp(-3.5, 3.5)
    x[0] *= 2.0 ** 65
    x[1] *= 2.0 ** 126                       # up to bf16's largest
    x[2, 0] = 2e19                           # one far head beside an ordinary one
    x[3] *= 2.0 ** 50                        # where the kernel's own scaling begins
    x[4, 0, 5], x[4, 0, 99] = float("inf"), float("-inf")
    x[5, 1, 127] = float("nan")
    x[T - 1, 1] *= 2.0 ** 100
    c.q = c.k = x.reshape(T, H * D).to(torch.bfloat16).cuda()
    q = c.call().view(T, H, D)
    torch.cuda.synchronize()
    k = torch.stack([c.kc[t // c.page, t % c.page] for t in range(T)])
    bad = torch.zeros((T, H), dtype=torch.bool)
    bad[4, 0] = bad[5, 1] = True
    for got, weight, scale, what in ((q, c.qw, c.qs, "q"), (k, c.kw, c.ks, "k")):
        lost = (got & 0x7F) == 0x7F if scale is not None else torch.isnan(got)
        assert bool(lost[bad].all()) and not bool(lost[~bad].any())
        with np.errstate(invalid="ignore"):  # the bad heads, which are not compared
            want, size = c.turned(c.k, weight)
        check_values(got[~bad], want[~bad.numpy()], size[~bad.numpy()], scale, what)


@pytest.mark.parametrize("pairs", [False, True])
def test_ties_at_position_0_go_to_the_even_code(pairs):
    """Where the rotation is the identity, a quotient can lie exactly between two codes. A tie needs
    a scale whose odd part fits a bf16 value's eight bits: all of them, against every value whose
    quotient lies in the codes' range, give the plain store's codes (none of these quotients lies
    within float32's error of a tie without being one: they differ by 1 / (31 * 255) or more)."""
    one = lambda x: torch.tensor([x], dtype=torch.float32, device="cuda")  # noqa: E731
    D, H = 128, 8
    tab = torch.cat([torch.ones((1, D // 2)), torch.zeros((1, D // 2))], dim=1).cuda()
    mant = np.arange(128, 256, dtype=np.float64)
    values = np.concatenate([mant * 2.0 ** e for e in range(-34, 4)])
    for odd in range(1, 256, 2):
        s = odd * 2.0 ** -12
        x = values[(values / s > 2.0 ** -11) & (values / s < 470)]
        x = np.concatenate([x, -x])
        T = -(-x.size // (H * D))
        x = torch.from_numpy(np.resize(x, (T, H * D))).to(torch.bfloat16).cuda()
        kc = torch.zeros((T, 1, H, D), dtype=torch.uint8, device="cuda")
        vc = torch.zeros_like(kc)
        q = fq.rope_kv_append(x, x, x, torch.zeros(T, dtype=torch.int64, device="cuda"), tab,
                              torch.arange(T, device="cuda"), kc, vc, interleaved=pairs,
                              q_scale=one(s), k_scale=one(s), v_scale=one(s))
        want = fq.quant_per_tensor(x, one(s))
        torch.cuda.synchronize()
        for got in (q, kc.view(T, -1), vc.view(T, -1)):
            assert torch.equal(got, want), s
