"""GPU parity of the experts' sort, dispatch, combine and combine's gradients against oracle.block.

The sort, the moved rows and dy (one float32 product, rounded once to the output type) must be equal
bit for bit. combine adds top_k float32 products: within (top_k + 1) half steps (2^-24) of the sum
of magnitudes, plus half a bf16 step (2^-8) of the value where it is rounded to bf16. dweights adds
N products: at most N / 32 + 64 additions follow one another.
"""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from oracle import block as ob
from tests.gpu_util import assert_within
from workloads import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


def choices(T, k, E, seed, kind="mixed"):
    rng = np.random.default_rng(seed)
    if kind == "one":      # every choice on one expert
        return np.full((T, k), E - 1)
    if kind == "none":     # no choice is this rank's
        return np.full((T, k), -1)
    if kind == "distinct":
        return np.argsort(rng.random((T, E)), axis=1)[:, :k]
    ids = rng.integers(0, E, (T, k))   # an expert may come twice in a row
    ids[rng.random((T, k)) < 0.2] = -1
    ids[rng.random((T, k)) < 0.05] = E
    ids[rng.random((T, k)) < 0.05] = E + 1000
    return ids


def check_sort(ids, E, dtype):
    t = torch.from_numpy(np.ascontiguousarray(ids)).to(dtype).cuda()
    off, rows, pos = fq.moe_sort(t, E)
    torch.cuda.synchronize()
    w_off, w_rows, w_pos = ob.moe_sort(ids, E)
    assert np.array_equal(off.cpu().numpy(), w_off)
    assert np.array_equal(pos.cpu().numpy(), w_pos)
    assert np.array_equal(rows.cpu().numpy(), w_rows)


# one workgroup (up to 16384 choices) and several, experts from one to the most
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (3, 2, 2), (64, 8, 128), (65, 7, 60),
                                   (1000, 8, 1024), (2048, 8, 128), (2049, 8, 128), (16385, 1, 3),
                                   (4096, 8, 128), (700, 64, 256), (9999, 6, 1024), (30000, 8, 17)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, k, E, dtype):
    print(f"[sort] T={T} k={k} E={E} {dtype}", flush=True)
    check_sort(choices(T, k, E, T + k), E, dtype)


@pytest.mark.parametrize("kind", ["one", "none"])
@pytest.mark.parametrize("T,k,E", [(5, 2, 4), (3000, 8, 64)])
def test_sort_crowded_and_empty(T, k, E, kind):
    check_sort(choices(T, k, E, 1, kind), E, torch.int64)


def test_sort_many_blocks():
    """Past 256 blocks of 8192 choices a block takes more; checked against torch's stable sort."""
    T, k, E = 300001, 8, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda")
    off, rows, pos = fq.moe_sort(ids, E)
    key = torch.where(ids >= 0, ids, E).view(-1)
    order = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    assert int(off[E]) == n
    assert torch.equal(rows[:n].long(), order[:n] // k) and bool((rows[n:] == -1).all())
    assert torch.equal(pos.view(-1)[order[:n]].long(), torch.arange(n, device="cuda"))
    assert torch.equal(torch.diff(off).long(), torch.bincount(key, minlength=E + 1)[:E])


def test_sort_extreme_ids_and_no_tokens():
    ids = torch.tensor([[2 ** 31 - 1, -2 ** 31], [1, 0]], dtype=torch.int32, device="cuda")
    off, rows, pos = fq.moe_sort(ids, 2)
    assert off.tolist() == [0, 1, 2] and rows.tolist() == [1, 1, -1, -1]
    assert pos.tolist() == [[-1, -1], [1, 0]]
    big = torch.tensor([[2 ** 32, -2 ** 62], [2 ** 32 + 1, 0]], device="cuda")
    off, rows, pos = fq.moe_sort(big, 2)
    assert off.tolist() == [0, 1, 1] and pos.tolist() == [[-1, -1], [-1, 0]]
    off = torch.full((5,), 9, dtype=torch.int32, device="cuda")
    off, rows, pos = fq.moe_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4,
                                 expert_offsets=off)
    assert off.tolist() == [0] * 5 and rows.numel() == 0 and pos.shape == (0, 2)


SHAPES = [(1, 1, 1, 8), (1, 8, 128, 2048), (5, 3, 4, 72), (64, 8, 128, 520), (37, 8, 16, 2048),
          (130, 2, 8, 4104), (33, 20, 30, 264), (257, 6, 60, 1032)]


def layout(T, k, E, seed):
    """pos of the sort and its rows, from a mix of local, repeated and foreign choices."""
    pos = ob.moe_sort(choices(T, k, E, seed), E)[2]
    return torch.from_numpy(pos).cuda(), T * k


@pytest.mark.parametrize("T,k,E,N", SHAPES)
def test_dispatch(T, k, E, N):
    print(f"[dispatch] T={T} k={k} E={E} N={N}", flush=True)
    pos, R = layout(T, k, E, 3)
    xb = synth.act_bf16(T, N + 8, seed=4).cuda()
    buf = torch.full((R, N + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    out = fq.moe_dispatch(xb[:, 8:], pos, out=buf[:, 8:8 + N])
    torch.cuda.synchronize()
    want = torch.full_like(buf, 3.0)
    p = pos.long().view(-1)
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    want[p[p >= 0], 8:8 + N] = xb[token[p >= 0], 8:]
    assert torch.equal(buf, want) and out.data_ptr() == buf[:, 8:].data_ptr()


@pytest.mark.parametrize("T,k,N", [(2100, 3, 136), (700, 5, 4104), (2048, 2, 2048), (2500, 1, 64)])
@pytest.mark.parametrize("lines", [True, False])
def test_dispatch_of_many_tokens(T, k, N, lines):
    """Rows that start on 128-byte lines and rows that do not, four chunks a lane."""
    print(f"[dispatch] T={T} k={k} N={N} lines={lines}", flush=True)
    pos, R = layout(T, k, 16, 33)
    x = synth.act_bf16(T, N, seed=34).cuda()
    pitch = -(-N // 64) * 64 + (0 if lines else 8)
    buf = torch.full((R, pitch), 3.0, dtype=torch.bfloat16, device="cuda")
    fq.moe_dispatch(x, pos, out=buf[:, :N])
    torch.cuda.synchronize()
    want = torch.full_like(buf, 3.0)
    p = pos.long().view(-1)
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    want[p[p >= 0], :N] = x[token[p >= 0]]
    assert torch.equal(buf, want)


@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,N", SHAPES)
def test_combine(T, k, E, N, y_dtype, o_dtype):
    print(f"[combine] T={T} k={k} E={E} N={N} {y_dtype} -> {o_dtype}", flush=True)
    pos, R = layout(T, k, E, 5)
    g = torch.Generator().manual_seed(6)
    yb = torch.randn((R, N + 8), generator=g).to(y_dtype).cuda()
    y = yb[:, 8:]
    for weighted in (True, False):
        w = torch.rand((T, k), generator=g).cuda() if weighted else None
        ob_ = torch.full((T, N + 8), 9.0, dtype=o_dtype, device="cuda")
        out = fq.moe_combine(y, pos, weights=w, out=ob_[:, :N])
        torch.cuda.synchronize()
        want, size = ob.moe_combine(f64(y), pos.cpu().numpy(), None if w is None else f64(w))
        bound = (k + 1) * U * size + (BF * np.abs(want) if o_dtype == torch.bfloat16 else 0)
        assert_within(f64(out), want, bound, "combine")
        assert bool((ob_[:, N:] == 9.0).all())
    fresh = fq.moe_combine(y, pos, weights=w, out_dtype=o_dtype)
    assert fresh.dtype == o_dtype and torch.equal(fresh, out)


@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,N", SHAPES)
def test_combine_backward(T, k, E, N, y_dtype):
    print(f"[combine bwd] T={T} k={k} E={E} N={N} {y_dtype}", flush=True)
    pos, R = layout(T, k, E, 7)
    g = torch.Generator().manual_seed(8)
    y = torch.randn((R, N), generator=g).to(y_dtype).cuda()
    dout = torch.randn((T, N), generator=g).to(torch.bfloat16).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    before = torch.full((R, N), 5.0, dtype=y_dtype, device="cuda")
    dy, dw = fq.moe_combine_bwd(dout, y, pos, weights=w, dy=before.clone())
    torch.cuda.synchronize()
    p = pos.long().view(-1)
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    want = before.clone()
    grads = (w.view(-1, 1) * dout[token].float()).to(y_dtype)
    want[p[p >= 0]] = grads[p >= 0]
    assert torch.equal(dy, want)
    d, size = ob.moe_dweights(f64(dout), f64(y), pos.cpu().numpy())
    assert_within(f64(dw), d, (N / 32 + 64) * U * size + 1e-40, "dweights")
    # in place of y, without weights, without y
    y2 = y.clone()
    dy2, dw2 = fq.moe_combine_bwd(dout, y2, pos, weights=w, dy=y2)
    torch.cuda.synchronize()
    assert torch.equal(dw2, dw)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[p[p >= 0]] = False
    assert torch.equal(y2[~keep], want[~keep]) and torch.equal(y2[keep], y[keep])
    dy3, none = fq.moe_combine_bwd(dout, None, pos, dy=before.clone())
    torch.cuda.synchronize()
    want[p[p >= 0]] = dout[token[p >= 0]].to(y_dtype)
    assert none is None and torch.equal(dy3, want)


def test_rows_past_the_end_are_left_out():
    """pos beyond the given rows: neither read nor written."""
    T, k, N, R = 4, 2, 64, 5
    pos = torch.tensor([[0, 7], [4, 5], [-3, 2], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32,
                       device="cuda")
    x = synth.act_bf16(T, N, seed=9).cuda()
    buf = torch.full((R + 3, N), 1.0, dtype=torch.bfloat16, device="cuda")
    fq.moe_dispatch(x, pos, out=buf[:R])
    want = torch.full_like(buf, 1.0)
    want[0], want[4], want[2] = x[0], x[1], x[2]
    assert torch.equal(buf, want)
    out = fq.moe_combine(buf[:R], pos)
    assert torch.equal(out[:3], x[:3]) and bool((out[3] == 0).all())
    buf2 = torch.full_like(buf, 1.0)
    dy, dw = fq.moe_combine_bwd(x, buf[:R], pos, dy=buf2[:R])
    assert torch.equal(buf2, want)
    assert dw[0, 1] == 0 and dw[1, 1] == 0 and bool((dw[3] == 0).all()) and dw[2, 0] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_no_choice_names_does_not_matter(dtype):
    """NaN and infinities in grouped rows that no choice names, and in the weights of choices without
    a row, reach nothing."""
    T, k, E, N = 70, 11, 6, 136
    pos, R = layout(T, k, E, 21)
    g = torch.Generator().manual_seed(22)
    y = torch.randn((R + 9, N), generator=g).to(dtype).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    dout = torch.randn((T, N), generator=g).to(torch.bfloat16).cuda()
    named = torch.zeros(R + 9, dtype=torch.bool, device="cuda")
    named[pos[pos >= 0].long()] = True
    assert not bool(named.all()) and bool((pos < 0).any())
    y2, w2 = y.clone(), w.clone()
    y2[~named] = float("nan")
    y2[R + 3] = float("inf")
    w2[pos < 0] = float("nan")
    dy = torch.zeros_like(y)
    for a, b in ((fq.moe_combine(y, pos, weights=w), fq.moe_combine(y2, pos, weights=w2)),
                 *zip(fq.moe_combine_bwd(dout, y, pos, weights=w, dy=dy.clone()),
                      fq.moe_combine_bwd(dout, y2, pos, weights=w2, dy=dy.clone()))):
        assert torch.equal(a, b) and bool(torch.isfinite(b).all())


def test_no_tokens_no_rows():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    pos0 = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    assert fq.moe_dispatch(e(0, 64), pos0).shape == (0, 64)
    assert fq.moe_combine(e(0, 64), pos0).shape == (0, 64)
    dy, dw = fq.moe_combine_bwd(e(0, 64), e(0, 64), pos0)
    assert dy.shape == (0, 64) and dw.shape == (0, 2)
    pos = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")  # tokens, but no grouped row
    out = fq.moe_combine(e(0, 64), pos, out=torch.full((3, 64), 4.0, device="cuda"))
    assert bool((out == 0).all())
    dy, dw = fq.moe_combine_bwd(torch.ones((3, 64), dtype=torch.bfloat16, device="cuda"), e(0, 64),
                                pos)
    torch.cuda.synchronize()
    assert dy.shape == (0, 64) and bool((dw == 0).all())


def test_rows_past_32_bit_offsets():
    """Grouped rows beyond 2^31 elements and 2^32 bytes of their buffer."""
    N = 4096
    R = (1 << 32) // (2 * N) + 70000
    y = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([[0, R - 1], [R - 40000, 7]], dtype=torch.int32, device="cuda")
    x = synth.act_bf16(2, N, seed=41).cuda()
    fq.moe_dispatch(x, pos, out=y)
    assert torch.equal(y[pos.long()], x[:, None, :].expand(2, 2, N))
    out = fq.moe_combine(y, pos, out_dtype=torch.float32)
    assert torch.equal(out, 2 * x.float())
    dout = synth.act_bf16(2, N, seed=42).cuda()
    _, dw = fq.moe_combine_bwd(dout, y, pos, dy=y)
    torch.cuda.synchronize()
    assert torch.equal(y[pos.long()], dout[:, None, :].expand(2, 2, N))
    want = (f64(dout) * f64(x)).sum(axis=1)
    size = np.abs(f64(dout) * f64(x)).sum(axis=1)
    assert_within(f64(dw), np.stack([want, want], 1), (N / 32 + 64) * U * np.stack([size, size], 1),
                  "far dweights")


def test_gradients_of_the_round_trip_against_differences():
    """loss = <combine(dispatch(x)), dout>: its gradient in x by combine of combine_bwd, in the
    weights by dweights, against the loss's exact dependence (it is bilinear)."""
    T, k, E, N = 6, 2, 3, 64
    pos, R = layout(T, k, E, 11)
    g = torch.Generator().manual_seed(12)
    x = torch.randn((T, N), generator=g).to(torch.bfloat16).cuda()
    dout = torch.randn((T, N), generator=g).to(torch.bfloat16).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    xg = fq.moe_dispatch(x, pos)
    dxg, dw = fq.moe_combine_bwd(dout, xg, pos, weights=w, dy=torch.zeros((R, N), device="cuda",
                                                                         dtype=torch.bfloat16))
    dx = fq.moe_combine(dxg, pos, out_dtype=torch.float32)
    torch.cuda.synchronize()
    W, X, D, live = f64(w), f64(x), f64(dout), (pos >= 0).cpu().numpy()

    def loss(X, W):
        return float(((W * live).sum(axis=1)[:, None] * X * D).sum())

    for t, n in ((0, 0), (3, 40), (5, 63)):
        e = np.zeros_like(X)
        e[t, n] = 1.0
        num = loss(X + e, W) - loss(X, W)
        # dxg is rounded to bf16 once for each choice
        assert abs(num - float(dx[t, n])) <= 2 * BF * (W * live).sum() * abs(D[t, n]) + 1e-9
    for t, j in ((0, 0), (2, 1), (5, 0)):
        e = np.zeros_like(W)
        e[t, j] = 1.0
        num = loss(X, W + e) - loss(X, W)
        assert abs(num - float(dw[t, j])) <= 1e-5 * np.abs(X[t] * D[t]).sum()


def test_sort_refuses_numbers_of_experts_out_of_range():
    """Past the C type, and at the ends of 64 bits, where E + 1 has no value."""
    ids = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    for E in (2 ** 63 - 1, -2 ** 63, 2 ** 31, -1):
        with pytest.raises(ValueError, match=f"E is {E}, out of range"):
            fq.moe_sort(ids, E, expert_offsets=torch.zeros(5, dtype=torch.int32, device="cuda"))
    for E in (0, 1025):
        with pytest.raises(fq.Fp8rlError):
            fq.moe_sort(ids, E)
    with pytest.raises(OverflowError):
        fq.moe_sort(ids, 2 ** 63, expert_offsets=torch.zeros(5, dtype=torch.int32, device="cuda"))


# one workgroup sorts up to 4096 choices, a tile of 256 in each of its 16 waves; more take two kernels
@pytest.mark.parametrize("T,k,E", [(513, 1, 128), (1025, 1, 128), (4095, 1, 128), (4096, 1, 128),
                                   (4097, 1, 128), (512, 8, 128), (513, 8, 128), (585, 7, 1024),
                                   (586, 7, 1024), (64, 64, 1), (65, 63, 1000), (257, 16, 17)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_around_a_full_workgroup(T, k, E, dtype):
    print(f"[sort] T={T} k={k} E={E} {dtype}", flush=True)
    blocks = -(-T * k // 4096)
    assert fq.fp8rl_moe_sort_workspace_bytes(T, k, E) == (4 * blocks * E if blocks > 1 else 0)
    check_sort(choices(T, k, E, T + k), E, dtype)
    check_sort(choices(T, k, E, T + k + 1, "one"), E, dtype)


def test_sort_at_the_most_blocks():
    """256 blocks of 4096 choices, and the first call past them, whose blocks take more."""
    E = 64
    for n in (256 * 4096, 256 * 4096 + 1):
        assert fq.fp8rl_moe_sort_workspace_bytes(n, 1, E) == 4 * 256 * E
        g = torch.Generator(device="cuda").manual_seed(n)
        ids = torch.randint(-1, E, (n, 1), generator=g, device="cuda")
        off, rows, pos = fq.moe_sort(ids, E)
        key = torch.where(ids >= 0, ids, E).view(-1)
        order = torch.sort(key, stable=True).indices
        m = int((key < E).sum())
        assert int(off[E]) == m
        assert torch.equal(rows[:m].long(), order[:m]) and bool((rows[m:] == -1).all())
        assert torch.equal(pos.view(-1)[order[:m]].long(), torch.arange(m, device="cuda"))
        assert bool((pos.view(-1)[order[m:]] == -1).all())
        assert torch.equal(torch.diff(off).long(), torch.bincount(key, minlength=E + 1)[:E])
