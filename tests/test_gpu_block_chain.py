"""The operators between the linears together with the linears, as a decoder block runs them, and
their behaviour under streams and graph capture.

Each stage is checked on the actual output of the stage before it (so that no tolerance has to cover
a chain of roundings), the mixture-of-experts layer also as a whole against the router's definition:
out[t] = sum_j weight[t][j] * expert_{id[t][j]}(x[t]).
"""

import numpy as np
import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from oracle import block as ob
from oracle import gemm as og
from oracle import quant as oq
from perf import operators as cases
from tests.gpu_util import assert_gemm_close, assert_within, bits16, gemm_out_to_f64
from tests.test_gpu_block_append import check_values
from tests.test_gpu_block_norm import check_bwd, check_norm
from workloads import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


def linear(N, K, seed):
    return fq.quant_weight(synth.weight_bf16(N, K, seed=seed).cuda())


def check_gemm(y, xq, sa, wq, sw, what):
    ref = og.gemm_blockscaled(xq.cpu().numpy(), sa.cpu().numpy(), wq.cpu().numpy(), sw.cpu().numpy(),
                              out="f64")
    rounded = og.bf16_bits_to_f64(og.round_f64_to_bf16_bits(ref))
    assert_gemm_close(gemm_out_to_f64(y), rounded, ref, "bf16", what)


@pytest.mark.parametrize("T", [1, 45])
def test_attention_side_of_a_block(T):
    """stream + delta -> norm codes -> q/k/v linear -> rotated append, all on one device queue."""
    K, Hq, Hkv, D, page = 512, 4, 2, 64, 16
    delta, stream = synth.act_bf16(T, K, seed=1).cuda(), synth.act_bf16(T, K, seed=2).cuda()
    w = (1 + 0.1 * torch.randn(K, generator=torch.Generator().manual_seed(3))).bfloat16().cuda()
    wq, sw = linear((Hq + 2 * Hkv) * D, K, 4)
    pos = torch.arange(100, 100 + T, device="cuda")
    ang = torch.arange(256, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(D // 2) / (D / 2))
    table = torch.cat([ang.cos(), ang.sin()], dim=1).float().cuda()
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(5))[:T].cuda()
    kc = torch.zeros((pages, page, Hkv, D), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    nw = torch.ones(D, dtype=torch.bfloat16, device="cuda")

    xq, sa, h, _ = fq.add_rmsnorm_quant(delta, w, residual=stream)
    qkv = fq.gemm(xq, sa, wq, sw)
    # scales from this batch's own largest values (of v; a normalised, rotated head stays below
    # sqrt(2 D))
    amax = torch.zeros(2, device="cuda")
    fq.amax(qkv[:, (Hq + Hkv) * D:], amax[1:])
    amax[0] = (2 * D) ** 0.5
    scale = fq.scale_from_amax(amax)
    q = fq.rope_kv_append(qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:],
                          pos, table, slots, kc, vc, q_weight=nw, k_weight=nw, k_scale=scale[0:1],
                          v_scale=scale[1:2])
    torch.cuda.synchronize()
    check_norm(delta, stream, w, 1e-6, (xq, sa, h, None), "norm")
    check_gemm(qkv, xq, sa, wq, sw, "qkv")
    cs = f64(table)[pos.cpu().numpy()]
    for name, lo, H, got, s in (("q", 0, Hq, q.view(T, Hq, D), None),
                                ("k", Hq * D, Hkv, kc[slots // page, slots % page], scale[0:1])):
        rows = f64(qkv[:, lo:lo + H * D]).reshape(-1, D)
        c = np.repeat(cs, H, axis=0)
        want, size = ob.rope(rows, np.ones(D), 1e-6, c[:, :D // 2], c[:, D // 2:], D, False)
        check_values(got, want.reshape(T, H, D), size.reshape(T, H, D), s, name)
    v = qkv[:, (Hq + Hkv) * D:]
    plain = fq.quant_per_tensor(v, scale[1:2])
    assert torch.equal(vc[slots // page, slots % page].reshape(T, Hkv * D), plain)


@pytest.mark.parametrize("T,away", [(1, False), (130, False), (130, True)])
def test_mixture_of_experts_layer(T, away):
    K, I, E, k = 256, 128, 8, 2
    delta, stream = synth.act_bf16(T, K, seed=11).cuda(), synth.act_bf16(T, K, seed=12).cuda()
    nw = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    router = torch.randn((E, K), generator=torch.Generator().manual_seed(13)).cuda()
    up = [linear(I, K, 20 + e) for e in range(E)]
    down = [linear(K, I, 40 + e) for e in range(E)]
    wq_u, sw_u = torch.stack([a for a, _ in up]), torch.stack([b for _, b in up])
    wq_d, sw_d = torch.stack([a for a, _ in down]), torch.stack([b for _, b in down])

    _, _, h, x = fq.add_rmsnorm_quant(delta, nw, residual=stream, rows=True)
    top = torch.topk(x.float() @ router.t(), k, dim=1)
    weights = torch.softmax(top.values, dim=1)
    ids = torch.where(top.indices % 2 == 1, -1, top.indices) if away else top.indices
    off, row_ids, pos = fq.moe_sort(ids, E)
    mid = fq.grouped_gemm_fused_act(x, wq_u, sw_u, off, row_ids=row_ids)
    y = fq.grouped_gemm_fused_act(torch.nn.functional.silu(mid), wq_d, sw_d, off)
    out = fq.moe_combine(y, pos, weights=weights)
    # the moved rows give the grouped GEMM the same bits as reading through row_ids
    n = int(off[E])
    moved = fq.moe_dispatch(x, pos, out=torch.zeros((T * k, K), dtype=torch.bfloat16, device="cuda"))
    mid2 = fq.grouped_gemm(*fq.quant_act(moved), wq_u, sw_u, off)
    torch.cuda.synchronize()
    assert torch.equal(mid2[:n], mid[:n])
    assert torch.equal(moved[:n], x[row_ids[:n].long()])

    # every token by itself, through the oracle's quantizer and GEMM
    xq, sa = oq.quant_act_tok128(bits16(x))
    W, chosen, rows = f64(weights), ids.cpu().numpy(), pos.cpu().numpy()
    ref_mid, ref_y = np.zeros((n, I)), np.zeros((n, K))
    for t in range(T):
        for j in range(k):
            e, r = int(chosen[t, j]), int(rows[t, j])
            assert (e < 0) == (r < 0)
            if e < 0:
                continue
            ref_mid[r] = og.gemm_blockscaled(xq[t:t + 1], sa[t:t + 1], wq_u[e].cpu().numpy(),
                                             sw_u[e].cpu().numpy(), out="f64")[0]
            aq, asc = oq.quant_act_tok128(bits16(torch.nn.functional.silu(mid[r:r + 1])))
            ref_y[r] = og.gemm_blockscaled(aq, asc, wq_d[e].cpu().numpy(), sw_d[e].cpu().numpy(),
                                           out="f64")[0]
    if n == 0:
        assert bool((out == 0).all())
        return
    for got, ref, what in ((mid[:n], ref_mid, "up"), (y[:n], ref_y, "down")):
        rounded = og.bf16_bits_to_f64(og.round_f64_to_bf16_bits(ref))
        assert_gemm_close(gemm_out_to_f64(got), rounded, ref, "bf16", what)
    want, size = ob.moe_combine(f64(y), rows, W)
    assert_within(f64(out), want, (k + 1) * U * size + BF * np.abs(want), "combine")
    # the layer as a whole: each expert's row within the GEMM's tolerance of the reference
    want, size = ob.moe_combine(ref_y, rows, W)
    slack = 1e-3 * np.sqrt(np.mean(ref_y ** 2)) * (W * (rows >= 0)).sum(axis=1)[:, None]
    assert_within(f64(out), want, 2.0 ** -7 * size + slack + BF * (size + slack), "layer")


def test_training_step_of_norm_and_experts():
    """Forward and backward of norm -> dispatch -> (a scale per expert) -> combine, gradients against
    differences of a float64 forward pass."""
    T, K, E, k, eps = 6, 128, 3, 2, 1e-3
    g = torch.Generator().manual_seed(31)
    x = torch.randn((T, K), generator=g).bfloat16().cuda()
    dout = torch.randn((T, K), generator=g).bfloat16().cuda()
    nw = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16().cuda()
    ids = torch.tensor([[0, 1], [2, 0], [1, -1], [2, 2], [0, 2], [1, 0]], device="cuda")
    wts = torch.rand((T, k), generator=g).cuda()
    gain = torch.tensor([0.5, 2.0, 1.0], device="cuda")  # the experts: exact factors

    off, row_ids, pos = fq.moe_sort(ids, E)
    n = int(off[E])
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.diff(off))
    _, _, _, y = fq.add_rmsnorm_quant(x, nw, codes=False, rows=True, eps=eps)
    zeros = lambda: torch.zeros((T * k, K), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    rows = fq.moe_dispatch(y, pos, out=zeros())
    rows[:n] *= gain[expert][:, None].bfloat16()
    out = fq.moe_combine(rows, pos, weights=wts)
    drows, dwts = fq.moe_combine_bwd(dout, rows, pos, weights=wts, dy=zeros())
    drows[:n] *= gain[expert][:, None].bfloat16()
    dy = fq.moe_combine(drows, pos)
    dx, dnw = fq.add_rmsnorm_bwd(dy, x, nw, eps=eps)
    torch.cuda.synchronize()
    check_bwd(dy, x, nw, None, eps, dx, dnw, "norm backward")

    X, NW, W, D = f64(x), f64(nw), f64(wts), f64(dout)
    G = np.where(ids.cpu().numpy() >= 0, f64(gain)[np.maximum(ids.cpu().numpy(), 0)], 0.0)

    def loss(X, NW, W):
        Y = X * NW / np.sqrt(np.mean(X * X, axis=1, keepdims=True) + eps)
        return float((((W * G).sum(axis=1)[:, None] * Y) * D).sum())

    # y, the moved rows' gradients and dy are each rounded to bf16: three half steps of what they
    # sum, and the differences' own error
    s = 1e-5
    for t, c in ((0, 0), (3, 77), (5, 127)):
        e = np.zeros_like(X)
        e[t, c] = s
        num = (loss(X + e, NW, W) - loss(X - e, NW, W)) / (2 * s)
        r = 1 / np.sqrt(np.mean(X[t] ** 2) + eps)
        mag = np.abs((W * G).sum(axis=1)[t] * D[t] * NW)
        size = r * (mag[c] + np.abs(X[t, c]) * r * r * np.mean(mag * np.abs(X[t])))
        assert abs(num - float(dx[t, c])) <= 4 * BF * size + 1e-5
    for c in (0, 64):
        e = np.zeros_like(NW)
        e[c] = s
        num = (loss(X, NW + e, W) - loss(X, NW - e, W)) / (2 * s)
        r = 1 / np.sqrt(np.mean(X ** 2, axis=1) + eps)
        assert abs(num - float(dnw[c])) <= 4 * BF * np.abs((W * G).sum(axis=1) * D[:, c] * X[:, c] * r).sum() + 1e-5
    for t, j in ((0, 1), (2, 0), (3, 1)):
        e = np.zeros_like(W)
        e[t, j] = s
        num = (loss(X, NW, W + e) - loss(X, NW, W - e)) / (2 * s)
        Yt = X[t] * NW / np.sqrt(np.mean(X[t] ** 2) + eps)
        assert abs(num - float(dwts[t, j])) <= 2 * BF * np.abs(G[t, j] * Yt * D[t]).sum() + 1e-5
    assert float(dwts[2, 1]) == 0.0
    assert bool(torch.isfinite(out).all())


SMALL = [
    dict(op="norm", M=70, K=2048, residual=True, rows=True),
    dict(op="norm_bwd", M=700, K=1152, stream=True),
    dict(op="sort", T=3000, E=60, top_k=4, N=520, rows=True, away=0.5, wide=True),  # two kernels
    dict(op="sort", T=40, E=60, top_k=4, N=520, rows=True, away=0.0, wide=False),
    dict(op="combine", T=100, E=16, top_k=5, N=1032, away=0.5, weighted=True, f32=False),
    dict(op="combine_bwd", T=100, E=16, top_k=5, N=1032, away=0.5, f32=True),
    dict(op="append", T=50, Hq=8, Hkv=2, D=128, rot=96, pairs=True, norms=True, cache8=True,
         q8=True, page=16, heads_first=True, pad=5),
]


def leaves(v):
    return {n: t.clone() for n, t in v.items()}


@pytest.fixture
def own():
    cases.own = True
    yield cases
    cases.own = False


@pytest.mark.parametrize("case", SMALL, ids=lambda c: c["op"] + str(c.get("T", c.get("M"))))
def test_graph_replays_equal_eager_on_new_inputs(case, own):
    """Captured once, replayed with other inputs written into the same tensors, eager work and
    synchronizations in between."""
    states = [own.prepare(case, s) for s in range(3)]
    want = [leaves(own.run(s)) for s in states]
    torch.cuda.synchronize()
    fresh = [own.prepare(case, s) for s in range(3)]
    static = own.prepare(case, 0)
    own.run(static)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = own.run(static)
    for rep in range(4):
        src = fresh[rep % 3]
        again = own.prepare(case, rep % 3)
        for n, t in again.items():
            if isinstance(t, torch.Tensor):
                static[n].copy_(t)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, t in want[rep % 3].items():
            assert torch.equal(out[n].view(torch.uint8) if t.element_size() == 1 else out[n],
                               t.view(torch.uint8) if t.element_size() == 1 else t), (rep, n)
        own.run(src)  # eager work between replays


@pytest.mark.parametrize("case", SMALL, ids=lambda c: c["op"] + str(c.get("T", c.get("M"))))
def test_two_graphs_and_a_side_stream(case, own):
    """Two graphs captured of the same calls replay in turn, and an eager pass on another stream
    beside them leaves both results alone."""
    a, b, c = (own.prepare(case, s) for s in (1, 2, 3))
    want = [leaves(own.run(own.prepare(case, s))) for s in (1, 2, 3)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(own.run(s))
        graphs.append(g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            third = own.run(c)
        graphs[1].replay()
    torch.cuda.synchronize()
    for got, w in zip(outs + [third], want):
        for n, t in w.items():
            x, y = (v.view(torch.uint8) if v.element_size() == 1 else v for v in (got[n], t))
            assert torch.equal(x, y), n


def test_stream_argument():
    """stream= runs the call there, with what it allocates."""
    side = torch.cuda.Stream()
    x = synth.act_bf16(600, 1024, seed=50).cuda()
    w = torch.ones(1024, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, 8, (2000, 4), device="cuda")
    torch.cuda.synchronize()
    a = fq.add_rmsnorm_quant(x, w, residual=x, stream=side)
    dx, dw = fq.add_rmsnorm_bwd(x, a[2], w, stream=side)
    off, rows, pos = fq.moe_sort(ids, 8, stream=side.cuda_stream)
    side.synchronize()
    b = fq.add_rmsnorm_quant(x, w, residual=x)
    ex, ew = fq.add_rmsnorm_bwd(x, b[2], w)
    want = fq.moe_sort(ids, 8)
    torch.cuda.synchronize()
    for p, q in zip(a[:3] + (dx, dw, off, rows, pos), b[:3] + (ex, ew) + want):
        assert torch.equal(p, q)
    with pytest.raises(ValueError):
        fq.add_rmsnorm_quant(x.cpu(), w, stream=side)
