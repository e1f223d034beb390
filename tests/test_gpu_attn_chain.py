"""Attention together with the operators around it, as a decoder block runs them, and its behaviour under
streams, graph capture and concurrent calls.

Each stage is checked on the actual output of the stage before it, with the tolerances of the stage's
own tests; two ways to the same attention are compared within the sum of their tolerances.
"""

import threading

import numpy as np
import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from oracle import attn as oa
from oracle import e4m3
from perf import more_operators as cases
from tests.gpu_util import assert_within
from tests.test_gpu_attn_decode import Paged, expected, f64, one, queries
from tests.test_gpu_attn_docs import BF, Docs, U, i32
from tests.test_gpu_block_chain import check_gemm, linear
from workloads import synth

pytestmark = pytest.mark.gpu


class Session:
    """Sequences whose tokens go through the q/k/v linear's output, the rotated append and attention:
    prompts first, then token by token."""

    def __init__(self, prompts, spare, *, Hq=4, Hkv=2, D=64, page=16, codes=True, seed=0):
        self.Hq, self.Hkv, self.D, self.page, self.codes = Hq, Hkv, D, page, codes
        self.lens, B = [0] * len(prompts), len(prompts)
        width = max(-(-(p + spare) // page) for p in prompts)
        rng = np.random.default_rng(seed)
        self.table = i32(rng.permutation(B * width + 1)[:B * width].reshape(B, width).tolist())
        kind = torch.uint8 if codes else torch.bfloat16
        self.kc, self.vc = (torch.zeros((B * width + 1, page, Hkv, D), dtype=kind, device="cuda")
                            for _ in range(2))
        self.scales = dict(k_scale=one(0.0131), v_scale=one(0.0117)) if codes else {}
        ang = torch.arange(4096, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(D // 2) / (D / 2))
        self.rotation = torch.cat([ang.cos(), ang.sin()], dim=1).float().cuda()

    def slots(self, new):
        """Positions and slots of `new[b]` more tokens of every sequence, and their q/k/v rows."""
        pos, slot = [], []
        for b, n in enumerate(new):
            j = torch.arange(self.lens[b], self.lens[b] + n, device="cuda")
            pos.append(j)
            slot.append(self.table[b].long()[j // self.page] * self.page + j % self.page)
            self.lens[b] += n
        return torch.cat(pos), torch.cat(slot)

    def append(self, rows, new):
        q, k, v = rows.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], dim=1)
        pos, slot = self.slots(new)
        return fq.rope_kv_append(q, k, v, pos, self.rotation, slot, self.kc, self.vc, **self.scales)

    def cached(self, b):
        """Keys and values of a sequence, float64 [n][Hkv][D]."""
        at = (self.table[b].long().repeat_interleave(self.page)[:self.lens[b]],
              torch.arange(self.lens[b], device="cuda") % self.page)
        out = []
        for x, c in (("k", self.kc), ("v", self.vc)):
            rows = c[at].cpu()
            out.append(e4m3.decode(rows.numpy()) * float(self.scales[x + "_scale"]) if self.codes
                       else f64(rows))
        return out


def rows_of(s, n, seed):
    return synth.act_bf16(n, (s.Hq + 2 * s.Hkv) * s.D, seed=seed).cuda()


def check_queries(s, b, q, got, positions, what, read_back=False):
    """got [n][Hq * D] against attention of q (as stored, float64) over what is cached. Codes that were
    read back are rounded to bf16: keys BF of their size, and so the scores, and values BF; the weights
    are rounded to bf16 there, by decode to 2^-11 (the bound for either cache)."""
    k, v = s.cached(b)
    j = np.arange(k.shape[0])
    for h in range(s.Hq):
        cols = slice(h * s.D, (h + 1) * s.D)
        kv = h * s.Hkv // s.Hq
        o, _, w, _, size, a = oa.attend(q[:, cols], k[:, kv], v[:, kv], positions, j,
                                        sm_scale=s.D ** -0.5)
        da = s.D * U * size.max() + 12 * U * np.abs(a).max()
        stored = BF if read_back and s.codes else 0.0
        rel = (2 * (da + stored * size.max()) + stored + (BF if read_back else 2.0 ** -11) + 20 * U
               + 2 * len(j) * U)
        assert_within(got[:, cols], o, BF * np.abs(o) + rel * (w @ np.abs(v[:, kv])), what)


@pytest.mark.parametrize("codes", [True, False])
def test_prompts_in_chunks_then_tokens(codes):
    """append, the cached prefix read back, a chunk's attention; then tokens by decode; all against
    the cache's own contents."""
    s = Session([70, 5, 130], 12, codes=codes)
    for step, new in enumerate(([40, 5, 100], [30, 0, 30])):
        q = s.append(rows_of(s, sum(new), seed=step), new)
        total = i32([0] + np.cumsum(s.lens).tolist())
        k, v = fq.kv_read(s.kc, s.vc, s.table, total, rows=sum(s.lens), **s.scales)
        starts = np.concatenate([[0], np.cumsum(new)])
        out, _ = fq.attn_fwd(q, k, v, s.D, i32(starts.tolist()), k_offsets=total)
        for b, n in enumerate(new):
            if n:
                at = slice(starts[b], starts[b + 1])
                check_queries(s, b, f64(q[at]), f64(out[at]), np.arange(s.lens[b] - n, s.lens[b]),
                              f"chunk {step} of {b}", read_back=True)
    wq, sw = linear(256, s.Hq * s.D, 9)
    for step in range(3):
        q = s.append(rows_of(s, 3, seed=10 + step), [1, 1, 1])
        out = fq.attn_decode(q, s.kc, s.vc, s.table, i32(s.lens), **s.scales)
        for b in range(3):
            check_queries(s, b, f64(q[b:b + 1]), f64(out[b:b + 1]), np.array([s.lens[b] - 1]),
                          f"token {step} of {b}")
        xq, sa = fq.quant_act(out)  # and on into the output linear
        check_gemm(fq.gemm(xq, sa, wq, sw), xq, sa, wq, sw, "output linear")


def test_decode_takes_the_appends_codes():
    s = Session([33], 1)
    s.append(rows_of(s, 33, seed=1), [33])
    rows = rows_of(s, 1, seed=2)
    q, k, v = rows.split([s.Hq * s.D, s.Hkv * s.D, s.Hkv * s.D], dim=1)
    pos, slot = s.slots([1])
    q8 = fq.rope_kv_append(q, k, v, pos, s.rotation, slot, s.kc, s.vc, q_scale=one(0.05), **s.scales)
    assert q8.dtype == torch.uint8
    out = fq.attn_decode(q8, s.kc, s.vc, s.table, i32(s.lens), q_scale=one(0.05), **s.scales)
    stored = e4m3.decode(q8.cpu().numpy()) * float(one(0.05))
    check_queries(s, 0, stored, f64(out), np.array([33]), "codes")


def test_one_token_chunks_are_decode():
    """A chunk of one query per sequence by either way."""
    s = Session([600, 40, 300], 0, codes=False)
    q = s.append(rows_of(s, 940, seed=3), [600, 40, 300])
    last = torch.tensor([599, 639, 939], device="cuda")
    total = i32([0, 600, 640, 940])
    k, v = fq.kv_read(s.kc, s.vc, s.table, total, rows=940)
    a, _ = fq.attn_fwd(q[last], k, v, s.D, i32([0, 1, 2, 3]), k_offsets=total, window=200)
    b = fq.attn_decode(q[last], s.kc, s.vc, s.table, i32(s.lens), window=200)
    worst = np.abs(f64(v)).max()
    assert np.abs(f64(a) - f64(b)).max() < 2 * (BF + BF) * worst


def all_four(state):
    """Append, decode, read, fwd and bwd on one state's buffers; their outputs."""
    s, d = state["session"], state["docs"]
    q = fq.rope_kv_append(*state["qkv"], state["pos"], s.rotation, state["slot"], s.kc, s.vc,
                          q_out=state["q_out"], **s.scales)
    out = fq.attn_decode(q, s.kc, s.vc, s.table, state["lens"], out=state["out"], **s.scales)
    fq.kv_read(s.kc, s.vc, s.table, state["offsets"], k_out=state["k"], v_out=state["v"], **s.scales)
    o, lse = d.fwd(out=state["o"], lse=state["lse"])
    grads = fq.attn_bwd(state["dout"], *d.dev, o, lse, d.D, d.q_offsets, dq=state["g"][0],
                        dk=state["g"][1], dv=state["g"][2], **d.args)
    return [out, state["k"], state["v"], o, lse, *grads]


def new_state(seed):
    s = Session([900, 30, 520], 8, seed=seed)
    s.append(rows_of(s, 1450, seed=seed), [900, 30, 520])
    d = Docs([90, 200, 33], D=64, seed=seed, before=0, behind=0)
    rows = rows_of(s, 3, seed=seed + 50)
    pos, slot = s.slots([1, 1, 1])
    bf = dict(dtype=torch.bfloat16, device="cuda")
    return dict(session=s, docs=d, pos=pos, slot=slot, lens=i32(s.lens), dout=d.dout.cuda(),
                qkv=[t.contiguous() for t in rows.split([256, 128, 128], dim=1)],
                q_out=torch.empty((3, 256), **bf), out=torch.empty((3, 256), **bf),
                offsets=i32([0, 10, 40, 200]), k=torch.zeros((200, 128), **bf),
                v=torch.zeros((200, 128), **bf), o=torch.zeros((d.Tq, 256), **bf),
                lse=torch.zeros((4, d.Tq), device="cuda"),
                g=[torch.zeros(t.shape, **bf) for t in (d.q, d.k, d.v)])


def test_graph_replays_equal_eager_calls():
    """One captured step, replayed on new inputs in the same buffers (other lengths among them), eager
    work and synchronizations between the replays."""
    state = new_state(1)
    all_four(state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = all_four(state)
    for round_ in range(4):
        other = new_state(2 + round_)
        if round_ % 2:
            other["lens"][0] = 17 + round_
        want = [t.clone() for t in all_four(other)]
        s, o = state["session"], other["session"]
        for a, b in ((s.kc, o.kc), (s.vc, o.vc), (s.table, o.table), (state["lens"], other["lens"]),
                     (state["pos"], other["pos"]), (state["slot"], other["slot"]),
                     (state["dout"], other["dout"]), *zip(state["qkv"], other["qkv"]),
                     *zip(state["docs"].dev, other["docs"].dev)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, want)):
            assert torch.equal(a, b), (round_, i)


def test_two_graphs_share_a_workspace():
    """Captured one after the other with the same memory, replayed in turn."""
    paged = Paged([2000, 700], 2, 64, seed=1)
    q, _ = queries(2, 4, 64, False, 2)
    ws = torch.empty(fq.fp8rl_attn_decode_workspace_bytes(2, 4, 2, 64, paged.table.shape[1] * 16),
                     dtype=torch.uint8, device="cuda")
    call = lambda w: fq.attn_decode(q, paged.raw["k"], paged.raw["v"], paged.dev_table,  # noqa: E731
                                    paged.dev_lens, window=w, workspace=ws, **paged.scales)
    want = [call(0).clone(), call(900).clone()]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for w in (0, 900):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(w))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        ws.fill_(255)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_on_another_stream():
    """Inputs made and used on a side stream, given as `stream` or as the current one."""
    state = new_state(7)
    want = [t.clone() for t in all_four(state)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    paged = Paged([1500, 90], 2, 64, seed=4)
    q, _ = queries(2, 4, 64, False, 5)
    args = (paged.raw["k"], paged.raw["v"], paged.dev_table, paged.dev_lens)
    ref = fq.attn_decode(q, *args, **paged.scales)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        late = torch.zeros_like(q)
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
        got = fq.attn_decode(late, *args, **paged.scales)
    given = torch.zeros_like(q)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        given.copy_(q)
    by_name = fq.attn_decode(given, *args, stream=side, **paged.scales)
    with torch.cuda.stream(side):
        again = [t.clone() for t in all_four(state)]
    side.synchronize()
    assert torch.equal(got, ref) and torch.equal(by_name, ref)
    for a, b in zip(again, want):
        assert torch.equal(a, b)


def test_two_calls_at_once():
    """Calls from two threads on streams of their own, each with its own workspace."""
    states = [new_state(20), new_state(21)]
    want = [[t.clone() for t in all_four(s)] for s in states]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got = all_four(states[i])
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                failed.append(i)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_a_training_step_by_autograd():
    """fwd and bwd inside a torch.autograd.Function, weights' gradients against float64 autograd of
    the same linear and attention."""
    class Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, offsets):
            out, lse = fq.attn_fwd(q, k, v, 32, offsets)
            ctx.save_for_backward(q, k, v, out, lse, offsets)
            return out

        @staticmethod
        def backward(ctx, dout):
            q, k, v, out, lse, offsets = ctx.saved_tensors
            return *fq.attn_bwd(dout.contiguous(), q, k, v, out, lse, 32, offsets), None

    g = torch.Generator().manual_seed(3)
    x = torch.randn((75, 64), generator=g).to(torch.bfloat16)
    w = (0.2 * torch.randn((3, 64, 64), generator=g)).to(torch.bfloat16)
    offsets = [0, 30, 75]
    wd = w.cuda().requires_grad_()
    q, k, v = (x.cuda() @ wd[i] for i in range(3))
    (Attention.apply(q, k, v, i32(offsets)).float() * x.cuda().float()).sum().backward()

    we = w.double().requires_grad_()
    qe, ke, ve = ((x.double() @ we[i]) for i in range(3))
    total = 0
    for a, b in zip(offsets, offsets[1:]):
        for h in range(2):
            c = slice(32 * h, 32 * h + 32)
            s = qe[a:b, c] @ ke[a:b, c].T / 32 ** 0.5
            s = s.masked_fill(torch.ones(b - a, b - a).triu(1).bool(), -torch.inf)
            total = total + (s.softmax(-1) @ ve[a:b, c] * x[a:b, c].double()).sum()
    total.backward()
    # products rounded to bf16 on the way in, gradients on the way out, P and dS between: a handful of
    # roundings, BF each of the size of the terms, which gradients of a few hundred terms average
    diff = f64(wd.grad) - we.grad.numpy()
    assert np.linalg.norm(diff) < 4 * BF * np.linalg.norm(we.grad.numpy())


@pytest.mark.parametrize("name", ["decode_one_stream", "read_prefixes", "fwd_short", "bwd_prefix"])
def test_listed_cases_agree_with_their_plain_forms(name):
    """The plain form and the framework's calls of one case each, on the same inputs."""
    case = next(c for c in cases.listed() if c["name"] == name)
    outs = []
    try:
        for cases.own in (False, True):
            out = cases.run(cases.prepare(case, 5))
            outs.append({k: f64(v) for k, v in out.items()})
    finally:
        cases.own = False
    for k in outs[0]:
        a, b = outs[0][k], outs[1][k]
        # two bf16 results of float32 sums, and the bf16 weights between: a few BF of the norm
        assert np.linalg.norm(a - b) <= 2 * BF * np.linalg.norm(a), k
