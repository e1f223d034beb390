"""The operators between the FP8 linears of a decoder block: their cases, their plain forms and the
framework's calls.

Four families, each a case's ``op``:

* ``norm`` / ``norm_bwd``: root-mean-square norm of the residual stream with the addition that
  produces it, the normalised rows leaving as E4M3 codes with one scale per 1x128 group (what the
  blockwise GEMM reads), and the norm's backward pass;
* ``sort``: the router's choices turned into the expert-ordered layout of the grouped GEMM
  (offsets, the token of every grouped row, the grouped row of every choice), with the rows moved
  there where ``rows`` asks for them;
* ``combine`` / ``combine_bwd``: the experts' rows weighted and summed per token, and the gradients
  of that sum;
* ``append``: rotation of q and k (after their per-head norms where the model has them) and the
  store of k and v into a paged cache in E4M3 or bf16.

``own`` false: elementary torch operations in float32, each result rounded once at the end. ``own``
true: the framework's calls.
"""

import math

import torch

own = False

BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # one new token of a single stream: the norm before a mixture-of-experts layer, whose
        # router reads the bf16 rows and whose experts read the codes
        dict(name="norm_one_token", op="norm", M=1, K=2048, residual=True, rows=True),
        # the norm before q/k/v at prefill of a 4096-wide dense model
        dict(name="norm_prefill", op="norm", M=8192, K=4096, residual=True, rows=False),
        # training: a short packed batch whose token count is no multiple of anything
        dict(name="norm_bwd_ragged", op="norm_bwd", M=1021, K=2048, stream=True),
        # training: a full micro-batch of a 4096-wide dense model
        dict(name="norm_bwd_train", op="norm_bwd", M=8192, K=4096, stream=True),
        # decode with 64 sequences: 128 experts, 8 per token, the grouped GEMM reads rows by index
        dict(name="sort_decode", op="sort", T=64, E=128, top_k=8, N=2048, rows=False, away=0.0,
             wide=True),
        # training: choices sorted and the rows moved, token count odd
        dict(name="sort_rows_train", op="sort", T=8191, E=128, top_k=8, N=2048, rows=True,
             away=0.0, wide=True),
        # decode with a ragged batch
        dict(name="combine_decode", op="combine", T=37, E=128, top_k=8, N=2048, away=0.0,
             weighted=True, f32=False),
        # prefill or a training step's forward pass
        dict(name="combine_prefill", op="combine", T=8192, E=128, top_k=8, N=2048, away=0.0,
             weighted=True, f32=False),
        # training: a short batch on one of two ranks that share the experts, so that half of the
        # choices are another rank's
        dict(name="combine_bwd_ranks", op="combine_bwd", T=509, E=128, top_k=8, N=2048, away=0.5,
             f32=False),
        # training: one layer of the mixture-of-experts model at its 4096 tokens
        dict(name="combine_bwd_train", op="combine_bwd", T=4096, E=128, top_k=8, N=2048, away=0.0,
             f32=False),
        # decode with 64 sequences: per-head norms, E4M3 cache of 16-token pages, q in bf16
        dict(name="append_decode", op="append", T=64, Hq=32, Hkv=8, D=128, rot=128, pairs=False,
             norms=True, cache8=True, q8=False, page=16, heads_first=False, pad=0),
        # prefill of a model without per-head norms, pages laid out head by head, q in E4M3 too,
        # a padded batch
        dict(name="append_prefill", op="append", T=8192, Hq=32, Hkv=8, D=128, rot=128, pairs=False,
             norms=False, cache8=True, q8=True, page=64, heads_first=True, pad=129),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "sort", "combine", "combine_bwd", "append"))
    if op in ("norm", "norm_bwd"):
        K = 128 * _log_int(rng, 8, 96)
        M = _log_int(rng, 1, max(1, 8192 * 4096 // max(K, 4096)))
        if op == "norm":
            rows = rng.random() < 0.4
            return dict(op=op, M=max(1, M * 5 // 7) if rows else M, K=K,
                        residual=rng.random() < 0.8, rows=rows)
        return dict(op=op, M=M, K=K, stream=rng.random() < 0.8)
    if op == "append":
        D = rng.choice((64, 80, 96, 128, 128, 256))
        Hkv = rng.choice((1, 2, 4, 8))
        Hq = Hkv * rng.choice((1, 2, 4, 7, 8))
        T = _log_int(rng, 1, max(1, 8192 * 48 * 128 // max(48 * 128, 2 * (Hq + 2 * Hkv) * D)))
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice((D, D, D // 2 // 16 * 16)),
                    pairs=rng.random() < 0.25, norms=rng.random() < 0.5, cache8=rng.random() < 0.7,
                    q8=rng.random() < 0.4, page=rng.choice((1, 16, 24, 64, 256)),
                    heads_first=rng.random() < 0.5, pad=rng.choice((0, 0, T // 8)))
    N = 8 * _log_int(rng, 64, 512)
    E = _log_int(rng, 4, 256)
    top_k = rng.randint(1, min(8, E))
    most = 4096 if op == "combine_bwd" else 8191
    T = _log_int(rng, 1, max(1, most * 8 * 2048 // max(8 * 2048, (top_k + 1) * N)))
    away = rng.choice((0.0, 0.0, 0.5, 0.75))
    if op == "sort":
        rows = rng.random() < 0.6
        T = T if rows else _log_int(rng, 1, 65536)
        return dict(op=op, T=T, E=E, top_k=top_k, N=N, rows=rows, away=away,
                    wide=rng.random() < 0.5)
    f32 = rng.random() < 0.2
    T = max(1, T // 2) if f32 else T
    if op == "combine":
        return dict(op=op, T=T, E=E, top_k=top_k, N=N, away=away, weighted=rng.random() < 0.8,
                    f32=f32)
    return dict(op=op, T=T, E=E, top_k=top_k, N=N, away=away, f32=f32)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["M"] * c["K"]
        each = 2 + (4 if c["residual"] else 0) + 1 + (2 if c["rows"] else 0)
        return {"bytes": n * each + n // 128 * 4 + 2 * c["K"], "flops": 7 * n}
    if c["op"] == "norm_bwd":
        n = c["M"] * c["K"]
        return {"bytes": n * (8 if c["stream"] else 6) + 6 * c["K"], "flops": 11 * n}
    if c["op"] == "append":
        q, kv = c["T"] * c["Hq"] * c["D"], 2 * c["T"] * c["Hkv"] * c["D"]
        out = q * (1 if c["q8"] else 2) + kv * (1 if c["cache8"] else 2)
        return {"bytes": 2 * (q + kv) + out + c["T"] * (4 * c["rot"] + 16),
                "flops": 5 * (q + kv)}
    n = c["T"] * c["top_k"]
    here = n * (1 - c["away"])  # rows that are this rank's
    if c["op"] == "sort":
        moved = 2 * c["N"] * (c["T"] + here) if c["rows"] else 0
        return {"bytes": n * ((8 if c["wide"] else 4) + 8) + 4 * (c["E"] + 1) + moved,
                "flops": 2 * n}
    b = 4 if c["f32"] else 2
    if c["op"] == "combine":
        return {"bytes": here * c["N"] * b + c["T"] * c["N"] * 2 + n * (8 if c["weighted"] else 4),
                "flops": 2 * here * c["N"]}
    return {"bytes": 2 * here * c["N"] * b + c["T"] * c["N"] * 2 + n * 12,
            "flops": 3 * here * c["N"]}


# ------------------------------------------------------------------------------------- the inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _stream_rows(g, M, K):
    """Rows of a residual stream: N(0, 1) with one channel in a hundred 20 times as large."""
    x = _randn(g, M, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 20
    return x.to(BF16)


def _choices(g, case):
    """Distinct experts per token, popular ones more often (rank r with weight r^-1.1); choices of
    another rank's experts are -1. The chosen experts' normalised weights beside them."""
    T, E, k = case["T"], case["E"], case["top_k"]
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)
    score = -1.1 * rank.float().log() - (-u.log()).log()
    top = torch.topk(score, k, dim=1)
    weights = torch.softmax(top.values, dim=1)
    ids = top.indices
    if case["away"]:
        gone = torch.randperm(E, generator=g, device="cuda")[:int(E * case["away"])]
        ids = torch.where(torch.isin(ids, gone), -1, ids)
    return ids, weights


def _sorted(ids, E):
    """Offsets, the token of every grouped row (-1 behind the last one) and the grouped row of
    every choice (-1 for another rank's), experts in order and each expert's choices in theirs."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    mine = (flat >= 0) & (flat < E)
    key = torch.where(mine, flat, E)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(counts[:E], 0)
    row = torch.arange(T * k, device=ids.device)
    pos = torch.empty_like(row)
    pos[order] = row
    pos = torch.where(mine, pos, -1).view(T, k)
    row_ids = torch.where(row < offsets[E], order // k, -1)
    return offsets.int(), row_ids.int(), pos.int()


def _rotation_table(positions, rot):
    """cos and sin of every position's angles, side by side, angles formed in 64 bits."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    angle = positions.double()[:, None] * 1e6 ** (-2 * i / max(rot, 1))
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] in ("norm", "norm_bwd"):
        M, K = c["M"], c["K"]
        s["weight"] = (1 + 0.2 * _randn(g, K)).to(BF16)
        if c["op"] == "norm":
            s["x"] = _stream_rows(g, M, K)
            s["residual"] = (3 * _stream_rows(g, M, K)) if c["residual"] else None
            s["h"] = torch.empty((M, K), dtype=BF16, device="cuda") if c["residual"] else None
            s["y"] = torch.empty((M, K), dtype=BF16, device="cuda") if c["rows"] else None
            s["xq"] = torch.empty((M, K), dtype=torch.uint8, device="cuda")
            s["sa"] = torch.empty((M, K // 128), dtype=torch.float32, device="cuda")
        else:
            s["h"] = _stream_rows(g, M, K)
            s["dy"] = (0.02 * _randn(g, M, K)).to(BF16)
            s["dh"] = (0.02 * _randn(g, M, K)).to(BF16) if c["stream"] else None
            s["dx"] = torch.empty((M, K), dtype=BF16, device="cuda")
            s["dw"] = torch.empty(K, dtype=torch.float32, device="cuda")
        return s
    if c["op"] == "append":
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        fused = _randn(g, T, (Hq + 2 * Hkv) * D).to(BF16)  # one GEMM's output: q, k and v columns
        s["q"] = fused[:, :Hq * D]
        s["k"] = fused[:, Hq * D:(Hq + Hkv) * D]
        s["v"] = fused[:, (Hq + Hkv) * D:]
        s["q_weight"] = (1 + 0.2 * _randn(g, D)).to(BF16) if c["norms"] else None
        s["k_weight"] = (1 + 0.2 * _randn(g, D)).to(BF16) if c["norms"] else None
        far = 32768
        s["table"] = _rotation_table(torch.arange(far, device="cuda"), c["rot"])
        s["positions"] = torch.randint(0, far, (T,), generator=g, device="cuda")
        pages = 2 * (-(-T // c["page"])) + 3
        slots = torch.randperm(pages * c["page"], generator=g, device="cuda")[:T].contiguous()
        if c["pad"]:
            slots[T - c["pad"]:] = -1  # rows behind the last sequence
        s["slots"] = slots
        shape = (pages, Hkv, c["page"], D) if c["heads_first"] else (pages, c["page"], Hkv, D)
        # what earlier calls left there
        cache = [torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)
                 if c["cache8"] else _randn(g, *shape).to(BF16) for _ in range(2)]
        # one view for both layouts: [page][place in the page][head][column]
        s["k_cache"], s["v_cache"] = ((t.transpose(1, 2) if c["heads_first"] else t) for t in cache)
        one = torch.ones(1, dtype=torch.float32, device="cuda")
        s["k_scale"], s["v_scale"] = (one * 0.0131, one * 0.0117) if c["cache8"] else (None, None)
        s["q_scale"] = one * 0.0142 if c["q8"] else None
        s["q_out"] = torch.empty((T, Hq * D), dtype=torch.uint8 if c["q8"] else BF16, device="cuda")
        return s
    T, E, k, N = c["T"], c["E"], c["top_k"], c["N"]
    ids, weights = _choices(g, c)
    if c["op"] == "sort":
        s["ids"] = ids.contiguous() if c["wide"] else ids.int()
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["row_ids"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
        s["pos"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        if c["rows"]:
            s["x"] = _stream_rows(g, T, N)
            s["moved"] = torch.zeros((T * k, N), dtype=BF16, device="cuda")
        return s
    kind = torch.float32 if c["f32"] else BF16
    s["pos"] = _sorted(ids, E)[2]
    s["y"] = _randn(g, T * k, N).to(kind)
    s["weights"] = weights.contiguous() if c.get("weighted", True) else None
    if c["op"] == "combine":
        s["out"] = torch.empty((T, N), dtype=BF16, device="cuda")
    else:
        s["dout"] = (0.02 * _randn(g, T, N)).to(BF16)
        s["dy"] = torch.zeros((T * k, N), dtype=kind, device="cuda")
        s["dweights"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------- one pass through an operator


def _codes(v):
    """E4M3 codes of float32 values, saturating."""
    return v.clamp(-448, 448).to(E4M3)


def _norm(s):
    c = s["case"]
    h = s["x"]
    if c["residual"]:
        h = (h.float() + s["residual"].float()).to(BF16)  # the stream as it is stored
    hf = h.float()
    y = hf * s["weight"].float() * torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS)
    groups = y.view(c["M"], c["K"] // 128, 128)
    amax = groups.abs().amax(2)
    sa = torch.where(amax == 0, 1.0, amax / 448)
    out = {"codes": _codes(groups / sa[:, :, None]).view(c["M"], c["K"]), "scales": sa}
    if c["residual"]:
        out["h"] = h
    if c["rows"]:
        out["y"] = y.to(BF16)
    return out


def _norm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    xhat = h * rstd
    gw = dy * s["weight"].float()
    dx = rstd * (gw - xhat * (gw * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(BF16), "dw": (dy * xhat).sum(0)}


def _sort(s):
    c = s["case"]
    offsets, row_ids, pos = _sorted(s["ids"], c["E"])
    out = {"offsets": offsets, "row_ids": row_ids, "pos": pos}
    if c["rows"]:
        rows = s["x"][row_ids.long().clamp(min=0)]
        out["moved"] = torch.where((row_ids >= 0)[:, None], rows, s["moved"])
    return out


def _combine(s):
    pos = s["pos"].long()
    rows = s["y"].float()[pos.clamp(min=0)]  # [T][k][N]
    w = (pos >= 0).float()
    if s["weights"] is not None:
        w = w * s["weights"]
    return {"out": (rows * w[:, :, None]).sum(1).to(BF16)}


def _combine_bwd(s):
    pos = s["pos"].long()
    T, k = pos.shape
    dout, mine = s["dout"].float(), pos >= 0
    dots = (s["y"].float()[pos.clamp(min=0)] * dout[:, None, :]).sum(2)
    grads = s["weights"][:, :, None] * dout[:, None, :]
    # every choice's gradient to its grouped row; those of other ranks to one row behind the end
    at = torch.where(mine, pos, T * k).view(-1)
    dy = torch.cat([s["dy"], s["dy"][:1]])
    dy[at] = grads.view(T * k, -1).to(dy.dtype)
    dy = dy[:T * k]
    return {"dy": dy, "dweights": torch.where(mine, dots, 0.0)}


def _head_norm(x, weight):
    return x * weight.float() * torch.rsqrt(x.square().mean(2, keepdim=True) + EPS)


def _rotate(x, cos, sin, rot, pairs):
    """x [T][H][D]: the first `rot` columns rotated, two halves against each other or, with
    `pairs`, each even column against the next."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2],
                                                            x[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], dim=3).flatten(2) if pairs else torch.cat([u, v], dim=2)
    return torch.cat([r, x[..., rot:]], dim=2)


def _stored(x, scale):
    return x.to(BF16) if scale is None else _codes(x / scale).view(torch.uint8)


def _append(s):
    c = s["case"]
    T, D, half = c["T"], c["D"], c["rot"] // 2
    at = s["table"][s["positions"]][:, None, :]
    cos, sin = at[..., :half], at[..., half:]
    q, k, v = (s[n].float().view(T, -1, D) for n in "qkv")
    if c["norms"]:
        q, k = _head_norm(q, s["q_weight"]), _head_norm(k, s["k_weight"])
    q = _stored(_rotate(q, cos, sin, c["rot"], c["pairs"]), s["q_scale"])
    k = _stored(_rotate(k, cos, sin, c["rot"], c["pairs"]), s["k_scale"])
    v = _stored(v, s["v_scale"])
    last = T - c["pad"]
    slots = s["slots"][:last]
    page, place = slots // c["page"], slots % c["page"]
    s["k_cache"][page, place] = k[:last]
    s["v_cache"][page, place] = v[:last]
    return _append_outputs(s, q.view(T, -1))


def _values(t):
    return t.view(E4M3) if t.dtype == torch.uint8 else t


def _append_outputs(s, q):
    heads_first = s["case"]["heads_first"]
    k, v = (t.transpose(1, 2) if heads_first else t for t in (s["k_cache"], s["v_cache"]))
    return {"q": _values(q), "k_cache": _values(k), "v_cache": _values(v)}


def _own_run(s):
    import fp8_blockwise_quantization_amd as fq

    c = s["case"]
    if c["op"] == "norm":
        xq, sa, h, y = fq.add_rmsnorm_quant(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                                            h=s["h"], y=s["y"], xq=s["xq"], sa=s["sa"])
        out = {"codes": xq.view(E4M3), "scales": sa}
        if c["residual"]:
            out["h"] = h
        if c["rows"]:
            out["y"] = y
        return out
    if c["op"] == "norm_bwd":
        dx, dw = fq.add_rmsnorm_bwd(s["dy"], s["h"], s["weight"], dh=s["dh"], eps=EPS, dx=s["dx"],
                                    dw=s["dw"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "sort":
        offsets, row_ids, pos = fq.moe_sort(s["ids"], c["E"], expert_offsets=s["offsets"],
                                            row_ids=s["row_ids"], pos=s["pos"])
        out = {"offsets": offsets, "row_ids": row_ids, "pos": pos}
        if c["rows"]:
            out["moved"] = fq.moe_dispatch(s["x"], pos, out=s["moved"])
        return out
    if c["op"] == "combine":
        return {"out": fq.moe_combine(s["y"], s["pos"], weights=s["weights"], out=s["out"])}
    if c["op"] == "combine_bwd":
        dy, dweights = fq.moe_combine_bwd(s["dout"], s["y"], s["pos"], weights=s["weights"],
                                          dy=s["dy"], dweights=s["dweights"])
        return {"dy": dy, "dweights": dweights}
    q = fq.rope_kv_append(s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"],
                          s["k_cache"], s["v_cache"], q_out=s["q_out"], interleaved=c["pairs"],
                          q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                          q_scale=s["q_scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _append_outputs(s, q)


def run(state):
    if own:
        return _own_run(state)
    plain = {"norm": _norm, "norm_bwd": _norm_bwd, "sort": _sort, "combine": _combine,
             "combine_bwd": _combine_bwd, "append": _append}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits


def _grid(v):
    """Values of the E4M3 grid nearest to v (ties to the even code), saturating, all in 64 bits."""
    m = v.abs()
    step = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * torch.clamp(torch.round(m / step) * step, max=448.0)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f = lambda t: t.to(torch.float64)  # noqa: E731
    if c["op"] == "norm":
        h = s["x"]
        if c["residual"]:
            h = (f(s["x"]) + f(s["residual"])).to(BF16)
        u = f(h)
        y = u * f(s["weight"]) / torch.sqrt((u * u).sum(1) / c["K"] + EPS)[:, None]
        parts = y.reshape(-1, 128)
        top = parts.abs().max(1).values
        scale = torch.where(top == 0, torch.ones_like(top), top / 448)
        out = {"codes": _grid(parts / scale[:, None]).reshape(y.shape),
               "scales": scale.reshape(c["M"], -1)}
        if c["residual"]:
            out["h"] = f(h)
        if c["rows"]:
            out["y"] = y
        return out
    if c["op"] == "norm_bwd":
        h, dy, w = f(s["h"]), f(s["dy"]), f(s["weight"])
        r = 1 / torch.sqrt((h * h).sum(1, keepdim=True) / c["K"] + EPS)
        lean = (dy * w * h).sum(1, keepdim=True) / c["K"]
        dx = r * w * dy - r ** 3 * lean * h
        if c["stream"]:
            dx = dx + f(s["dh"])
        return {"dx": dx, "dw": torch.mv((dy * h).t().contiguous(), r[:, 0])}
    if c["op"] == "sort":
        if not c["rows"]:
            return None  # whole numbers alone
        moved, at = f(s["moved"]), 0
        for e in range(c["E"]):
            token = torch.nonzero(s["ids"] == e)[:, 0]
            moved[at:at + len(token)] = f(s["x"][token])
            at += len(token)
        return {"offsets": None, "row_ids": None, "pos": None, "moved": moved}
    if c["op"] in ("combine", "combine_bwd"):
        pos = s["pos"].long()
        w = f(s["weights"]) if s["weights"] is not None else torch.ones_like(f(pos))
        outs = torch.zeros((c["T"], c["N"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros((c["T"], c["top_k"]), dtype=torch.float64, device="cuda")
        dy = f(s["dy"]) if c["op"] == "combine_bwd" else None
        for j in range(c["top_k"]):
            t = torch.nonzero(pos[:, j] >= 0)[:, 0]
            rows = f(s["y"][pos[t, j]])
            if dy is None:
                outs[t] += w[t, j, None] * rows
            else:
                dw[t, j] = (rows * f(s["dout"][t])).sum(1)
                dy[pos[t, j]] = w[t, j, None] * f(s["dout"][t])
        return {"out": outs} if dy is None else {"dy": dy, "dweights": dw}
    T, D, rot = c["T"], c["D"], c["rot"]
    even = torch.arange(0, rot, 2, device="cuda") if c["pairs"] else torch.arange(rot // 2,
                                                                                  device="cuda")
    odd = even + (1 if c["pairs"] else rot // 2)
    angle = f(s["table"])[s["positions"]]
    turn = torch.complex(angle[:, :rot // 2], angle[:, rot // 2:])[:, None, :]

    def heads(x, weight, rotated, scale):
        x = f(x).reshape(T, -1, D)
        if weight is not None:
            x = x * f(weight) / torch.sqrt((x * x).sum(2, keepdim=True) / D + EPS)
        if rotated:
            z = torch.complex(x[..., even], x[..., odd]) * turn
            x = x.clone()
            x[..., even], x[..., odd] = z.real, z.imag
        return x if scale is None else _grid(x / f(scale))

    q = heads(s["q"], s["q_weight"], True, s["q_scale"])
    out = {"q": q.reshape(T, -1)}
    for n, weight, rotated in (("k", s["k_weight"], True), ("v", None, False)):
        x = heads(s[n], weight, rotated, s[n + "_scale"])
        cache = f(_values(s[n + "_cache"]))
        last = T - c["pad"]
        slots = s["slots"][:last]
        cache[slots // c["page"], slots % c["page"]] = x[:last]
        out[n + "_cache"] = cache.transpose(1, 2) if c["heads_first"] else cache
    return out
