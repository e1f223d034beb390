"""GPU parity of the norm with codes and of its backward pass against oracle.block (float64).

Tolerances count float32 roundings (half a step: 2^-24) and the final rounding of the result's type
(bf16: 2^-8 of the value):
* a row's sum of squares is added over at most 128 values per lane, 6 steps across a wave and 16
  across waves, all terms positive: with the mean's and eps's roundings at most 154 of them, halved
  by the square root; the reciprocal square root is within 2 half steps and the products that
  follow add 3: r, and what is proportional to it, is within R = 82 half steps of exact;
* dx adds a mean of signed terms (the same 154) and three products to that: 256 half steps of the
  sum of its terms' magnitudes;
* dw adds M rows: at most M / 256 + 64 additions follow one another, and each term carries r's error:
  M / 256 + 160 half steps of the sum of magnitudes.
Codes with float32 scales are those of exact quotients and must be equal.
"""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from oracle import block as ob
from oracle import e4m3
from tests.gpu_util import assert_within
from workloads import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
R = 82 * U


def f64(t):
    return t.detach().double().cpu().numpy()


def stream_rows(M, K, seed):
    return synth.act_bf16(M, K, seed=seed)


def weights(K, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.2 * torch.randn(K, generator=g)).to(torch.bfloat16)


def check_norm(x, res, w, eps, out, what):
    xq, sa, h, y = out
    torch.cuda.synchronize()
    wh, wy = ob.add_rmsnorm(f64(x), None if res is None else f64(res), f64(w), eps)
    if h is not None:
        assert np.array_equal(f64(h), wh), what
    if y is not None:
        assert_within(f64(y), wy, (BF + 2 * R) * np.abs(wy) + 1e-40, what + " y")
    if xq is not None:
        codes, S = ob.quant_rows(wh, f64(w), wy)
        bad = np.nonzero(xq.cpu().numpy() != codes)
        assert bad[0].size == 0, (what, bad[0][:4], bad[1][:4])
        assert_within(f64(sa), S, R * S, what + " scales")


# one row up to many, one group up to the widest row, chunks that do not fill the threads; with the
# row counts at which lanes are dealt out differently
SHAPES = [(2, 4096), (8, 2048), (6, 1024), (3, 640), (8193, 1024), (8200, 1152), (8192, 2048), (600, 2176), (530, 5120), (2100, 512),
          (8200, 128), (4100, 256), (700, 1024), (1, 128), (1, 2048), (3, 4096), (64, 4096), (5, 384), (130, 2176), (33, 5120), (7, 8192),
          (9, 11008), (4, 16384), (3, 20480), (2, 32768), (1500, 2048), (2111, 4096), (4099, 1152),
          (1100, 7168)]


@pytest.mark.parametrize("M,K", SHAPES)
def test_norm_with_residual_codes_and_rows(M, K):
    print(f"[norm] {M}x{K}", flush=True)
    x, res = stream_rows(M, K, 1).cuda(), stream_rows(M, K, 2).cuda()
    w = weights(K, 3).cuda()
    out = fq.add_rmsnorm_quant(x, w, residual=res, rows=True)
    check_norm(x, res, w, 1e-6, out, f"{M}x{K}")


@pytest.mark.parametrize("M,K", [(1, 128), (5, 4096), (257, 2048), (1030, 4096)])
def test_norm_without_residual_and_single_outputs(M, K):
    x, w = stream_rows(M, K, 4).cuda(), weights(K, 5).cuda()
    full = fq.add_rmsnorm_quant(x, w, rows=True, eps=1e-5)
    check_norm(x, None, w, 1e-5, full, "no residual")
    assert full[2] is None
    only_codes = fq.add_rmsnorm_quant(x, w, eps=1e-5)
    only_rows = fq.add_rmsnorm_quant(x, w, eps=1e-5, codes=False, rows=True)
    torch.cuda.synchronize()
    assert only_codes[3] is None and only_rows[0] is None and only_rows[1] is None
    for a, b in ((only_codes[0], full[0]), (only_codes[1], full[1]), (only_rows[3], full[3])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,K", [(6, 256), (70, 4096), (1200, 2048)])
def test_norm_pitches_slices_and_places(M, K):
    """Rows inside wider buffers, h in place of the residual and of x; what lies around stays."""
    g = torch.Generator().manual_seed(6)
    wide = lambda cols: torch.randn((M, cols), generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    xb, rb, yb, hb = wide(K + 64), wide(K + 8), wide(K + 16), wide(K + 24)
    x, res, y, h = xb[:, 32:32 + K], rb[:, 8:], yb[:, 8:8 + K], hb[:, 16:16 + K]
    qb = torch.full((M, K + 32), 0x5A, dtype=torch.uint8, device="cuda")
    xq = qb[:, 16:16 + K]
    w = weights(K, 7).cuda()
    around = [t.clone() for t in (xb, rb, yb, hb)]
    out = fq.add_rmsnorm_quant(x, w, residual=res, y=y, xq=xq, h=h)
    check_norm(x, res, w, 1e-6, out, "slices")
    assert torch.equal(xb, around[0]) and torch.equal(rb, around[1])
    assert torch.equal(yb[:, :8], around[2][:, :8]) and torch.equal(yb[:, 8 + K:], around[2][:, 8 + K:])
    assert torch.equal(hb[:, :16], around[3][:, :16]) and torch.equal(hb[:, 16 + K:], around[3][:, 16 + K:])
    assert bool((qb[:, :16] == 0x5A).all()) and bool((qb[:, 16 + K:] == 0x5A).all())
    ref = [t.clone() for t in (out[0], out[1], out[2])]
    for place in (0, 1):
        a, b = x.clone(), res.clone()
        got = fq.add_rmsnorm_quant(a, w, residual=b, h=(a, b)[place])
        torch.cuda.synchronize()
        assert got[2].data_ptr() == (a, b)[place].data_ptr()
        for p, q in zip(got[:3], ref):
            assert torch.equal(p, q)


def test_norm_rows_past_32_bit_offsets():
    """Rows 2^30 elements apart: the fourth begins past 2^32 bytes."""
    K, ld, M = 256, 1 << 30, 4
    big = torch.empty((M - 1) * ld + K, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((M, K), (ld, 1))
    x.copy_(stream_rows(M, K, 50))
    w = weights(K, 51).cuda()
    res = stream_rows(M, K, 52).cuda()
    check_norm(x.clone(), res, w, 1e-6, fq.add_rmsnorm_quant(x, w, residual=res, h=res.clone(),
                                                            y=torch.empty_like(res)), "far")
    dy = stream_rows(M, K, 53).cuda()
    dx, dw = fq.add_rmsnorm_bwd(dy, x, w)
    check_bwd(dy, x.clone(), w, None, 1e-6, dx, dw, "far")
    want = dx.clone()
    far = fq.add_rmsnorm_bwd(dy, x.clone(), w, dx=x)[0]
    torch.cuda.synchronize()
    assert torch.equal(far, want)


def test_norm_edge_rows():
    """Zero rows and groups, one huge value, tiny values, rows that are not finite."""
    K = 512
    x = torch.zeros((8, K))
    x[1, 5] = 3.0                      # three groups of zeros beside one value
    x[2] = 1e-20                       # eps decides
    x[3] = torch.linspace(-448, 448, K)
    x[4, 100] = 1e15
    x[5] = 1.0
    x = x.to(torch.bfloat16).cuda()
    w = weights(K, 8).cuda()
    w[7] = 0.0
    check_norm(x[:6], None, w, 1e-6, fq.add_rmsnorm_quant(x[:6], w, rows=True), "edge")
    sa = fq.add_rmsnorm_quant(x, w)[1]
    assert bool((sa[0] == 1).all()) and bool((sa[1, 1:] == 1).all())
    bad = x.clone()
    bad[6, 3], bad[7, 9] = float("inf"), float("nan")
    bad[5, 0] = 2.0 ** 100             # its square is past float32
    for scale in ("fp32", "pow2"):
        xq, sa, _, y = fq.add_rmsnorm_quant(bad, w, rows=True, scale=scale)
        good = fq.add_rmsnorm_quant(x, w, rows=True, scale=scale)
        torch.cuda.synchronize()
        assert bool(torch.isnan(sa[5:]).all()) and bool(torch.isnan(y[5:]).all())
        assert torch.equal(sa[:5], good[1][:5]) and torch.equal(xq[:5], good[0][:5])


@pytest.mark.parametrize("M,K", [(3, 256), (65, 4096), (1300, 2048)])
def test_norm_power_of_two_scales(M, K):
    """Scales are powers of two with 448 S within the float32 error of max|y| or above it and S / 2
    below, and codes the nearest to y / S (half an E4M3 step, plus r's error)."""
    x, res, w = stream_rows(M, K, 9).cuda(), stream_rows(M, K, 10).cuda(), weights(K, 11).cuda()
    xq, sa, h, y = fq.add_rmsnorm_quant(x, w, residual=res, scale="pow2")
    torch.cuda.synchronize()
    wh, wy = ob.add_rmsnorm(f64(x), f64(res), f64(w), 1e-6)
    S = f64(sa)
    assert np.all(np.frexp(S)[0] == 0.5)
    top = np.abs(wy).reshape(M, K // 128, 128).max(axis=2)
    assert np.all(448 * S >= top * (1 - 2 * R)) and np.all(224 * S < top * (1 + 2 * R))
    v = wy / np.repeat(S, 128, axis=1)
    got = e4m3.decode(xq.cpu().numpy())
    bound = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 2 * R * np.abs(v)
    assert_within(got, np.clip(v, -448, 448), bound, "pow2 codes")
    # a lone value on the border: 448 is 448 * 2^0 exactly, one step above needs the next power
    xb = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    xb[0, 0], xb[1, 0] = 1.0, 1.0
    one = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    sb = fq.add_rmsnorm_quant(xb, one, scale="pow2", eps=1e-6)[1]
    assert float(sb[0, 0]) == 2.0 ** -5  # y = sqrt(128) = 11.3 <= 448 / 32 = 14, > 7


def test_norm_codes_feed_the_gemm():
    """The GEMM on the codes equals the GEMM on the dequantized values within its tolerance."""
    from oracle import gemm as og
    from oracle import quant as oq
    from tests.gpu_util import assert_gemm_close, bits16, gemm_out_to_f64

    M, K, N = 70, 512, 256
    x, res, w = stream_rows(M, K, 12).cuda(), stream_rows(M, K, 13).cuda(), weights(K, 14).cuda()
    xq, sa, _, _ = fq.add_rmsnorm_quant(x, w, residual=res)
    wt = synth.weight_bf16(N, K, seed=15)
    wq, sw = fq.quant_weight(wt.cuda())
    y = fq.gemm(xq, sa, wq, sw, out_dtype=torch.float32)
    torch.cuda.synchronize()
    rwq, rsw = oq.quant_weight_blk128(bits16(wt))
    ref = og.gemm_blockscaled(xq.cpu().numpy(), sa.cpu().numpy(), rwq, rsw, out="f64")
    assert_gemm_close(gemm_out_to_f64(y), ref, ref, "f32", "norm -> gemm")


def test_empty_norm():
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    w = weights(256, 1).cuda()
    xq, sa, h, _ = fq.add_rmsnorm_quant(x, w, residual=x)
    assert xq.shape == (0, 256) and sa.shape == (0, 2) and h.shape == (0, 256)
    dx, dw = fq.add_rmsnorm_bwd(x, x, w, dw=torch.full((256,), 7.0, device="cuda"))
    torch.cuda.synchronize()
    assert dx.shape == (0, 256) and bool((dw == 0).all())


# ---------------------------------------------------------------------------------------- backward


def check_bwd(dy, h, w, dh, eps, dx, dw, what):
    torch.cuda.synchronize()
    wx, ww, sx, sw = ob.add_rmsnorm_bwd(f64(dy), f64(h), f64(w), None if dh is None else f64(dh), eps)
    assert_within(f64(dx), wx, BF * np.abs(wx) + 256 * U * sx + 1e-40, what + " dx")
    if dw is not None:
        assert_within(f64(dw), ww, (dy.shape[0] / 256 + 160) * U * sw + 1e-40, what + " dw")


@pytest.mark.parametrize("M,K", SHAPES)
def test_norm_backward(M, K):
    print(f"[norm bwd] {M}x{K}", flush=True)
    g = torch.Generator().manual_seed(20)
    dy = (0.1 * torch.randn((M, K), generator=g)).to(torch.bfloat16).cuda()
    dh = (0.1 * torch.randn((M, K), generator=g)).to(torch.bfloat16).cuda()
    h, w = stream_rows(M, K, 21).cuda(), weights(K, 22).cuda()
    dx, dw = fq.add_rmsnorm_bwd(dy, h, w, dh=dh)
    check_bwd(dy, h, w, dh, 1e-6, dx, dw, f"{M}x{K}")
    dx0, none = fq.add_rmsnorm_bwd(dy, h, w, weight_grad=False)
    assert none is None
    check_bwd(dy, h, w, None, 1e-6, dx0, None, f"{M}x{K} no stream gradient")
    again = fq.add_rmsnorm_bwd(dy, h, w, dh=dh)
    torch.cuda.synchronize()
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)  # the same bits


@pytest.mark.parametrize("M,K", [(5, 256), (40, 4096), (700, 2048), (1500, 4224)])
def test_norm_backward_in_place_and_pitches(M, K):
    g = torch.Generator().manual_seed(23)
    big = torch.randn((M, 3 * K + 8), generator=g).to(torch.bfloat16).cuda()
    dy, dh, h = big[:, :K], big[:, K + 8:2 * K + 8], big[:, 2 * K + 8:]
    w = weights(K, 24).cuda()
    ref = fq.add_rmsnorm_bwd(dy, h, w, dh=dh)
    check_bwd(dy, h, w, dh, 1e-6, ref[0], ref[1], "slices")
    for place in (0, 1):
        a, b = dy.clone(), dh.clone()
        dx, dw = fq.add_rmsnorm_bwd(a, h, w, dh=b, dx=(a, b)[place])
        torch.cuda.synchronize()
        assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])


@pytest.mark.parametrize("M", [1, 2, 8, 600])
def test_norm_backward_dw_of_any_alignment(M):
    """dw that begins between 16-byte steps (a single workgroup's sums would be stored there)."""
    K = 1024
    dy, h, w = stream_rows(M, K, 60).cuda(), stream_rows(M, K, 61).cuda(), weights(K, 62).cuda()
    want = fq.add_rmsnorm_bwd(dy, h, w)[1]
    for shift in (1, 2, 3):
        buf = torch.full((K + 8,), 5.0, device="cuda")
        fq.add_rmsnorm_bwd(dy, h, w, dw=buf[shift:shift + K])
        torch.cuda.synchronize()
        assert torch.equal(buf[shift:shift + K], want)
        assert bool((buf[:shift] == 5).all()) and bool((buf[shift + K:] == 5).all())


def test_norm_backward_against_differences():
    """The gradients against central differences of the forward pass in float64."""
    M, K, eps, s = 4, 128, 1e-3, 1e-5
    g = torch.Generator().manual_seed(25)
    dy, dh, h = (torch.randn((M, K), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    w = weights(K, 26).cuda()
    dx, dw = fq.add_rmsnorm_bwd(dy, h, w, dh=dh, eps=eps)
    torch.cuda.synchronize()
    H, W, DY, DH = f64(h), f64(w), f64(dy), f64(dh)

    def loss(H, W):
        return float((H * W / np.sqrt(np.mean(H * H, axis=1, keepdims=True) + eps) * DY).sum()
                     + (H * DH).sum())

    for m, k in ((0, 0), (1, 64), (3, 127)):
        e = np.zeros_like(H)
        e[m, k] = s
        num = (loss(H + e, W) - loss(H - e, W)) / (2 * s)
        # the difference is off by s^2 times a third derivative of order 1; bf16 by 2^-8
        assert abs(num - float(dx[m, k])) <= BF * abs(num) + 1e-4
    for k in (0, 33, 127):
        e = np.zeros_like(W)
        e[k] = s
        num = (loss(H, W + e) - loss(H, W - e)) / (2 * s)
        assert abs(num - float(dw[k])) <= 1e-4 * (1 + abs(num))


def test_a_workspace_that_does_not_fit_raises_torchs_error():
    """As torch.empty would: the type that a caller who frees memory and tries again looks for."""
    M, K = 1025, 32768
    dy, h, w = stream_rows(M, K, 70).cuda(), stream_rows(M, K, 71).cuda(), weights(K, 72).cuda()
    dx, dw = torch.empty_like(dy), torch.empty(K, device="cuda")
    need = fq.fp8rl_add_rmsnorm_bwd_workspace_bytes(M, K)
    assert need == 32 << 20
    want = [t.clone() for t in fq.add_rmsnorm_bwd(dy, h, w, dx=dx, dw=dw)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction(torch.cuda.memory_reserved() / total)
    held = []
    try:
        with pytest.raises(torch.OutOfMemoryError):
            while len(held) < 10000:  # what torch still holds of free memory
                held.append(torch.empty(need, dtype=torch.uint8, device="cuda"))
        with pytest.raises(torch.OutOfMemoryError):
            fq.add_rmsnorm_bwd(dy, h, w, dx=dx, dw=dw)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    del held
    dx.zero_()
    got = fq.add_rmsnorm_bwd(dy, h, w, dx=dx, dw=dw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
