"""Attention of a decoder block, over the paged cache and over packed rows: its cases, its plain forms
and the framework's calls.

Four operators, each a case's ``op``:

* ``decode``: one new token of every sequence against the paged cache (bf16 or E4M3);
* ``read``: cached keys and values of ragged sequences back as contiguous bf16 rows;
* ``fwd``: packed documents' queries against their keys, with the statistic that training keeps;
* ``bwd``: the gradients of that.

Query i of a document with Lq queries and Lk keys is at position p = i + Lk - Lq; it sees key j if
(not causal or j <= p) and (no window or p - j < window), or if j < prefix. Its scores are
a = cap tanh(s / cap) - slope |p - j| with s = q.k / sqrt(D) (s itself without a cap).

``own`` false: elementary torch operations in float32, each result rounded once at the end. ``own``
true: the framework's calls.
"""

import math
import random

import torch

own = False

BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # a single stream a few hundred tokens in: latency counts
        dict(name="decode_one_stream", op="decode", B=1, Hq=32, Hkv=8, D=128, L=477, pad=0,
             cache8=True, q8=False, page=16, heads_first=False, window=0, cap=0.0, bias=False),
        # decode with 64 sequences of all lengths up to 4096, E4M3 cache of 16-token pages
        dict(name="decode_batch", op="decode", B=64, Hq=32, Hkv=8, D=128, L=4096, pad=0,
             cache8=True, q8=False, page=16, heads_first=False, window=0, cap=0.0, bias=False),
        # a few long contexts of the mixture-of-experts model, bf16 cache, pages head by head
        dict(name="decode_long", op="decode", B=8, Hq=32, Hkv=4, D=128, L=32768, pad=0,
             cache8=False, q8=False, page=64, heads_first=True, window=0, cap=0.0, bias=False),
        # wide heads with capped scores and a sliding window, a batch padded for graph replay
        dict(name="decode_window", op="decode", B=37, Hq=16, Hkv=8, D=256, L=6000, pad=3,
             cache8=True, q8=True, page=24, heads_first=False, window=1024, cap=50.0, bias=False),
        # a few cached prefixes read back before their next chunk of prompt
        dict(name="read_prefixes", op="read", B=3, Hkv=8, D=128, T=1021, cache8=True, page=16,
             heads_first=False, pad=7),
        # the prefixes of a full prefill batch
        dict(name="read_batch", op="read", B=16, Hkv=8, D=128, T=32768, cache8=True, page=64,
             heads_first=True, pad=0),
        # a few short prompts packed together
        dict(name="fwd_short", op="fwd", docs=5, Hq=32, Hkv=8, D=128, Tq=509, past=0, pad=3,
             causal=True, window=0, prefix=0, cap=0.0, bias=False),
        # prefill of one long prompt
        dict(name="fwd_prefill", op="fwd", docs=1, Hq=32, Hkv=8, D=128, Tq=8192, past=0, pad=0,
             causal=True, window=0, prefix=0, cap=0.0, bias=False),
        # the next chunk of prompts whose beginnings are cached, capped scores, the first keys
        # always seen beside a window
        dict(name="fwd_chunk", op="fwd", docs=4, Hq=16, Hkv=4, D=64, Tq=2048, past=4096, pad=0,
             causal=True, window=1024, prefix=64, cap=30.0, bias=False),
        # training: a short packed batch, bias by distance and prefixes seen by all
        dict(name="bwd_prefix", op="bwd", docs=7, Hq=16, Hkv=4, D=64, Tq=1021, past=0, pad=5,
             causal=True, window=0, prefix=96, cap=0.0, bias=True),
        # training: the mixture-of-experts model's 4096 tokens as a few packed documents
        dict(name="bwd_docs", op="bwd", docs=6, Hq=32, Hkv=4, D=128, Tq=4096, past=0, pad=0,
             causal=True, window=0, prefix=0, cap=0.0, bias=False),
        # training: one long document
        dict(name="bwd_train", op="bwd", docs=1, Hq=32, Hkv=8, D=128, Tq=8192, past=0, pad=0,
             causal=True, window=0, prefix=0, cap=0.0, bias=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("decode", "read", "fwd", "bwd"))
    Hkv = rng.choice((1, 2, 4, 8))
    D = rng.choice((64, 80, 96, 128, 128))
    if op in ("decode", "read"):
        D = rng.choice((D, D, 256))
        c = dict(op=op, Hkv=Hkv, D=D, cache8=rng.random() < 0.6,
                 page=rng.choice((1, 16, 24, 64, 256)), heads_first=rng.random() < 0.5)
        if op == "read":
            T = _log_int(rng, 1, 32768 * 1024 // max(1024, 2 * Hkv * D))
            return dict(c, B=_log_int(rng, 1, min(T, 64)), T=T, pad=rng.choice((0, 0, 13)))
        B = _log_int(rng, 1, 256)
        L = _log_int(rng, 1, min(32768, max(64, (1 << 27) // (B * Hkv * D))))
        return dict(c, B=B, L=L, Hq=Hkv * rng.choice((1, 2, 4, 7, 8)), q8=rng.random() < 0.4,
                    pad=rng.choice((0, 0, B // 8)), window=rng.choice((0, 0, _log_int(rng, 1, 4096))),
                    cap=rng.choice((0.0, 0.0, 30.0, 50.0)), bias=rng.random() < 0.25)
    Hq = Hkv * rng.choice((1, 2, 4, 7, 8))
    most = int(math.sqrt((8192 * 8192 if op == "fwd" else 4096 * 8192) * 32 / max(Hq, 8)))
    Tq = _log_int(rng, 1, min(8192, most))
    past = rng.choice((0, 0, rng.randint(0, max(0, min(most * most // Tq, 16384) - Tq)))
                      ) if op == "fwd" else 0
    return dict(op=op, docs=_log_int(rng, 1, min(Tq, 32)), Hq=Hq, Hkv=Hkv, D=D, Tq=Tq, past=past,
                pad=rng.choice((0, 0, 17)), causal=rng.random() < 0.8,
                window=rng.choice((0, 0, _log_int(rng, 1, 2048))),
                prefix=rng.choice((0, 0, _log_int(rng, 1, 512))),
                cap=rng.choice((0.0, 0.0, 20.0, 50.0)), bias=rng.random() < 0.25)


def _parts(total, n, least):
    """n whole numbers of at least `least` with that sum, uneven; the same for the same arguments."""
    rng = random.Random(total * 1009 + n)
    cuts = sorted(rng.randint(0, total - n * least) for _ in range(n - 1))
    return [b - a + least for a, b in zip([0] + cuts, cuts + [total - n * least])]


def _lengths(c):
    """Cached tokens of every sequence of a decode batch, the longest L; 0 for rows of padding."""
    rng = random.Random(c["L"] * 1009 + c["B"])
    least = c["L"] - c["L"] // 16 if c["B"] <= 8 else 1
    lens = [c["L"]] + [rng.randint(least, c["L"]) for _ in range(c["B"] - c["pad"] - 1)]
    return lens + [0] * (c["B"] - len(lens))


def _documents(c):
    """Queries and keys of every document."""
    nq = _parts(c["Tq"], c["docs"], 1)
    return nq, [a + b for a, b in zip(nq, _parts(c["past"], c["docs"], 0))]


def _visible(p, n, c):
    """How many of n keys the query at position p sees."""
    hi = min(p + 1, n) if c["causal"] else n
    lo = max(0, p - c["window"] + 1) if c["window"] else 0
    pre = min(c["prefix"], n)
    return pre + max(0, hi - max(lo, pre))


def work(case):
    c = case
    kv = 2 * c["Hkv"] * c["D"]  # values of a token's keys and values
    if c["op"] == "read":
        return {"bytes": c["T"] * kv * ((1 if c["cache8"] else 2) + 2), "flops": c["T"] * kv}
    if c["op"] == "decode":
        keys = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
        q = c["B"] * c["Hq"] * c["D"]
        return {"bytes": keys * kv * (1 if c["cache8"] else 2) + q * (3 if c["q8"] else 4),
                "flops": 4 * keys * c["Hq"] * c["D"]}
    nq, nk = _documents(c)
    pairs = sum(_visible(i + b - a, b, c) for a, b in zip(nq, nk) for i in range(a))
    q, k = c["Tq"] * c["Hq"] * c["D"], sum(nk) * kv
    if c["op"] == "fwd":
        return {"bytes": 4 * q + 2 * k + 4 * c["Tq"] * c["Hq"], "flops": 4 * pairs * c["Hq"] * c["D"]}
    return {"bytes": 8 * q + 4 * k + 4 * c["Tq"] * c["Hq"], "flops": 10 * pairs * c["Hq"] * c["D"]}


# ------------------------------------------------------------------------------------- the inputs


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(g, c, lens, s):
    """Caches whose pages are dealt out at random, the page table, the scales: N(0, 1) keys and
    values everywhere, in places that no sequence has as well."""
    need = [-(-n // c["page"]) for n in lens]
    pages, width = sum(need) + 3, max(max(need), 1)
    shape = (pages, c["Hkv"], c["page"], c["D"]) if c["heads_first"] else (pages, c["page"],
                                                                           c["Hkv"], c["D"])
    one = torch.ones(1, dtype=torch.float32, device="cuda")
    s["k_scale"], s["v_scale"] = (one * 0.0131, one * 0.0117) if c["cache8"] else (None, None)
    for n in "kv":
        t = _randn(g, *shape)
        t = (t / s[n + "_scale"]).clamp_(-448, 448).to(E4M3).view(torch.uint8) if c["cache8"] \
            else t.to(BF16)
        s[n + "_cache"] = t.transpose(1, 2) if c["heads_first"] else t
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(width, device="cuda")[None, :] < _int32(need)[:, None]
    table[used] = torch.randperm(pages, generator=g, device="cuda")[:sum(need)].int()
    s["table"] = table


def _offsets(lens):
    return _int32([0] + [sum(lens[:i + 1]) for i in range(len(lens))])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    D = c["D"]
    if c["op"] == "read":
        lens = _parts(c["T"], c["B"], 1)
        # every sequence's rows begin a little after its first cached token
        starts = [n % 37 for n in lens]
        _cache(g, c, [a + b for a, b in zip(lens, starts)], s)
        s["offsets"], s["starts"] = _offsets(lens), _int32(starts)
        shape = (c["T"] + c["pad"], c["Hkv"] * D)
        s["k_out"] = torch.ones(shape, dtype=BF16, device="cuda")
        s["v_out"] = torch.ones(shape, dtype=BF16, device="cuda")
        return s
    s["slopes"] = torch.exp2(-8 * (torch.arange(c["Hq"], device="cuda") + 1) / c["Hq"]).float() \
        if c["bias"] else None
    if c["op"] == "decode":
        lens = _lengths(c)
        order = torch.randperm(len(lens) - c["pad"], generator=g, device="cuda").tolist()
        lens = [lens[i] for i in order] + [0] * c["pad"]
        _cache(g, c, lens, s)
        s["lengths"] = _int32(lens)
        q = _randn(g, c["B"], c["Hq"] * D)
        s["q_scale"] = torch.full((1,), 0.0142, device="cuda") if c["q8"] else None
        s["q"] = (q / s["q_scale"]).clamp_(-448, 448).to(E4M3).view(torch.uint8) if c["q8"] \
            else q.to(BF16)
        s["out"] = torch.empty((c["B"], c["Hq"] * D), dtype=BF16, device="cuda")
        return s
    nq, nk = _documents(c)
    s["q_offsets"], s["k_offsets"] = _offsets(nq), _offsets(nk)
    s["prefix"] = torch.full((c["docs"],), c["prefix"], dtype=torch.int32, device="cuda") \
        if c["prefix"] else None
    Tq, Tk, Hq, Hkv = sum(nq) + c["pad"], sum(nk) + c["pad"], c["Hq"], c["Hkv"]
    if c["past"]:
        s["q"] = _randn(g, Tq, Hq * D).to(BF16)
        s["k"], s["v"] = _randn(g, Tk, Hkv * D).to(BF16), _randn(g, Tk, Hkv * D).to(BF16)
    else:  # one linear's output: q, k and v columns
        fused = _randn(g, Tq, (Hq + 2 * Hkv) * D).to(BF16)
        s["q"], s["k"], s["v"] = (t for t in fused.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    s["out"] = torch.zeros((Tq, Hq * D), dtype=BF16, device="cuda")
    s["lse"] = torch.zeros((Hq, Tq), dtype=torch.float32, device="cuda")
    if c["op"] == "bwd":
        s["out"], s["lse"] = _fwd(s).values()
        s["dout"] = (0.02 * _randn(g, Tq, Hq * D)).to(BF16)
        # the linear's output gradient: dq, dk and dv columns
        grads = torch.zeros((Tq, (Hq + 2 * Hkv) * D), dtype=BF16, device="cuda")
        s["dq"], s["dk"], s["dv"] = (t for t in grads.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    return s


# ------------------------------------------------------------------- one pass through an operator


def _stored(t, scale):
    """Stored values (bf16, or E4M3 codes and their scale) as float32."""
    return t.float() if scale is None else t.view(E4M3).float() * scale


def _cached(cache, table, scale):
    """Every sequence's cached rows in order, [B][heads][keys][D]; places without a page hold some
    other row."""
    rows = _stored(cache, scale)[table.long().clamp(min=0)]  # [B][pages][places][heads][D]
    return rows.flatten(1, 2).transpose(1, 2)


def _read(s):
    c = s["case"]
    row = torch.arange(c["T"], device="cuda")
    b = (row[:, None] >= s["offsets"][None, 1:]).sum(1)
    at = s["starts"].long()[b] + row - s["offsets"].long()[b]
    page = s["table"].long()[b, at // c["page"]]
    out = {}
    for n in "kv":
        rows = _stored(s[n + "_cache"][page, at % c["page"]], s[n + "_scale"])
        out[n] = torch.cat([rows.flatten(1).to(BF16), s[n + "_out"][c["T"]:]])
    return out


def _scores(raw, distance, seen, c, slopes):
    """Scores a of raw products, [..., queries, keys] with the heads at dim -3; -inf where the key
    is not seen."""
    a = raw * (1 / math.sqrt(c["D"]))
    if c["cap"]:
        a = torch.tanh(a / c["cap"]) * c["cap"]
    if slopes is not None:
        a = a - slopes[:, None, None] * distance.abs()
    return torch.where(seen, a, -math.inf)


def _weights(a):
    """exp(a - max), its sum and the max, over the last dim; a row without keys has the sum 0."""
    top = a.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(a - top)
    return p, p.sum(-1, keepdim=True), top


def _decode(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    k, v = (_cached(s[n + "_cache"], s["table"], s[n + "_scale"]) for n in "kv")
    q = _stored(s["q"], s["q_scale"]).view(B, Hkv, Hq // Hkv, D)
    raw = torch.matmul(q, k.transpose(2, 3)).view(B, Hq, 1, -1)
    last = s["lengths"][:, None, None, None] - 1
    distance = last - torch.arange(k.shape[2], device="cuda")
    seen = distance >= 0
    if c["window"]:
        seen = seen & (distance < c["window"])
    p, total, _ = _weights(_scores(raw, distance, seen, c, s["slopes"]))
    p = (p / total.clamp(min=1e-30)).view(B, Hkv, Hq // Hkv, -1)
    return {"out": torch.matmul(p, v).reshape(B, Hq * D).to(BF16)}


def _places(offsets, rows, back):
    """The document of every row (one past the last for rows of padding) and its place in it,
    `back` rows further on."""
    row = torch.arange(rows, device="cuda")
    doc = (row[:, None] >= offsets[None, 1:]).sum(1)
    last = len(offsets) - 2
    at = doc.clamp(max=last)
    return doc, row - offsets[at] + back[at]


def _mask(s):
    """Distances p - j and whether key j is seen, [queries][keys]."""
    c = s["case"]
    nq, nk = s["q_offsets"].diff(), s["k_offsets"].diff()
    dq, p = _places(s["q_offsets"], s["q"].shape[0], nk - nq)
    dk, j = _places(s["k_offsets"], s["k"].shape[0], 0 * nk)
    distance = p[:, None] - j[None, :]
    seen = torch.ones_like(distance, dtype=torch.bool)
    if c["causal"]:
        seen = seen & (distance >= 0)
    if c["window"]:
        seen = seen & (distance < c["window"])
    if c["prefix"]:
        seen = seen | (j < c["prefix"])[None, :]
    here = (dq < c["docs"])[:, None] & (dq[:, None] == dk[None, :])
    return distance, seen & here, dq < c["docs"]


def _heads(t, D):
    return t.float().view(t.shape[0], -1, D).transpose(0, 1)


def _products(x, y):
    """x [Hq][n][D] against y [Hkv][m][D]: [Hq][n][m], a head of y shared by Hq / Hkv of x."""
    shared = x.reshape(y.shape[0], -1, x.shape[2])
    return torch.matmul(shared, y.transpose(1, 2)).view(x.shape[0], x.shape[1], -1)


def _rows(t):
    return t.transpose(0, 1).flatten(1)


def _fwd(s):
    c = s["case"]
    q, k, v = (_heads(s[n], c["D"]) for n in "qkv")
    distance, seen, real = _mask(s)
    p, total, top = _weights(_scores(_products(q, k), distance, seen, c, s["slopes"]))
    out = _rows(_products(p, v.transpose(1, 2).contiguous()) / total.clamp(min=1e-30)).to(BF16)
    return {"out": torch.where(real[:, None], out, s["out"]),
            "lse": torch.where(real, (total.log() + top)[..., 0], s["lse"])}


def _bwd(s):
    c = s["case"]
    q, k, v, do, o = (_heads(s[n], c["D"]) for n in ("q", "k", "v", "dout", "out"))
    Hkv, keys = k.shape[0], k.shape[1]
    distance, seen, real = _mask(s)
    a = _scores(_products(q, k), distance, seen, c, s["slopes"])
    p = torch.exp(a - s["lse"][..., None])
    ds = p * (_products(do, v) - (do * o).sum(-1, keepdim=True))
    if c["cap"]:
        if s["slopes"] is not None:
            a = a + s["slopes"][:, None, None] * distance.abs()
        ds = torch.where(seen, ds * (1 - (a / c["cap"]).square()), 0.0)
    ds = ds * (1 / math.sqrt(c["D"]))
    dq = _products(ds, k.transpose(1, 2).contiguous())
    # the heads that share a key head: their rows one below the other
    dk = torch.matmul(ds.view(Hkv, -1, keys).transpose(1, 2), q.reshape(Hkv, -1, c["D"]))
    dv = torch.matmul(p.view(Hkv, -1, keys).transpose(1, 2), do.reshape(Hkv, -1, c["D"]))
    return {n: torch.where(real[:, None], _rows(t).to(BF16), s[n])
            for n, t in (("dq", dq), ("dk", dk), ("dv", dv))}


def _own_run(s):
    import fp8_blockwise_quantization_amd as fq

    c = s["case"]
    if c["op"] == "read":
        k, v = fq.kv_read(s["k_cache"], s["v_cache"], s["table"], s["offsets"], starts=s["starts"],
                          k_scale=s["k_scale"], v_scale=s["v_scale"], k_out=s["k_out"],
                          v_out=s["v_out"])
        return {"k": k, "v": v}
    if c["op"] == "decode":
        return {"out": fq.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                                      window=c["window"], cap=c["cap"], slopes=s["slopes"],
                                      q_scale=s["q_scale"], k_scale=s["k_scale"],
                                      v_scale=s["v_scale"], out=s["out"])}
    mask = dict(causal=c["causal"], window=c["window"], prefix=s["prefix"], cap=c["cap"],
                slopes=s["slopes"])
    if c["op"] == "fwd":
        out, lse = fq.attn_fwd(s["q"], s["k"], s["v"], c["D"], s["q_offsets"],
                               k_offsets=s["k_offsets"], out=s["out"], lse=s["lse"], **mask)
        return {"out": out, "lse": lse}
    dq, dk, dv = fq.attn_bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], c["D"],
                             s["q_offsets"], k_offsets=s["k_offsets"], dq=s["dq"], dk=s["dk"],
                             dv=s["dv"], **mask)
    return {"dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _own_run(state)
    plain = {"read": _read, "decode": _decode, "fwd": _fwd, "bwd": _bwd}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits


def _f64(t, scale=None):
    t = t.view(E4M3) if t.dtype == torch.uint8 else t
    return t.to(torch.float64) * (1.0 if scale is None else scale.to(torch.float64))


def _one_head(q, k, p, j, pre, c, slope):
    """The weights of one head of one document and the derivative of the capped score, in 64
    bits. q [n][D] at positions p, k [m][D]."""
    gap = p[:, None] - j[None, :]
    no = torch.zeros_like(gap, dtype=torch.bool)
    if c.get("causal", True):
        no |= gap < 0
    if c["window"]:
        no |= gap >= c["window"]
    no &= j[None, :] >= pre
    s = torch.mm(q, k.t()) / c["D"] ** 0.5
    slant = 1.0
    if c["cap"]:
        e = torch.expm1(-2 * s.abs() / c["cap"])
        tanh = -e / (2 + e) * torch.sign(s)
        s, slant = c["cap"] * tanh, 1 - tanh * tanh
    if slope is not None:
        s = s - slope * gap.abs()
    s = s.masked_fill(no, -math.inf)
    lse = torch.logsumexp(s, 1)
    w = torch.where(no, 0.0, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[:, None]))
    return w, slant, lse


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    D = c["D"]
    if c["op"] in ("read", "decode"):
        paged = {}
        lens = (s["offsets"].diff() + s["starts"] if c["op"] == "read" else s["lengths"]).tolist()
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            page = s["table"][b].long()[torch.div(j, c["page"], rounding_mode="floor")]
            for x in "kv":
                paged[b, x] = _f64(s[x + "_cache"][page, j % c["page"]], s[x + "_scale"])
        if c["op"] == "read":
            out = {x: _f64(s[x + "_out"]) for x in "kv"}
            for b, start in enumerate(s["starts"].tolist()):
                lo, hi = s["offsets"][b:b + 2].tolist()
                for x in "kv":
                    out[x][lo:hi] = paged[b, x][start:].reshape(hi - lo, -1)
            return out
        q = _f64(s["q"], s["q_scale"]).view(c["B"], c["Hq"], D)
        out = torch.zeros_like(q)
        group = c["Hq"] // c["Hkv"]
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            for h in range(c["Hq"] if n else 0):
                slope = None if s["slopes"] is None else s["slopes"][h].double()
                k, v = paged[b, "k"][:, h // group], paged[b, "v"][:, h // group]
                w, _, _ = _one_head(q[b, h:h + 1], k, j[-1:], j, 0, c, slope)
                out[b, h] = torch.mv(v.t(), w[0])
        return {"out": out.view(c["B"], -1)}
    nq, nk = _documents(c)
    group = c["Hq"] // c["Hkv"]
    wanted = ("out", "lse") if c["op"] == "fwd" else ("dq", "dk", "dv")
    out = {n: _f64(s[n]).clone() for n in wanted}
    for b in range(c["docs"]):
        rq = slice(sum(nq[:b]), sum(nq[:b + 1]))
        rk = slice(sum(nk[:b]), sum(nk[:b + 1]))
        j = torch.arange(nk[b], device="cuda")
        p = torch.arange(nq[b], device="cuda") + nk[b] - nq[b]
        for h in range(c["Hq"]):
            cq = slice(h * D, (h + 1) * D)
            ck = slice(h // group * D, (h // group + 1) * D)
            q, k, v = _f64(s["q"][rq, cq]), _f64(s["k"][rk, ck]), _f64(s["v"][rk, ck])
            slope = None if s["slopes"] is None else s["slopes"][h].double()
            w, slant, lse = _one_head(q, k, p, j, c["prefix"], c, slope)
            if c["op"] == "fwd":
                out["out"][rq, cq] = torch.mm(w, v)
                out["lse"][h, rq] = lse
                continue
            do = _f64(s["dout"][rq, cq])
            dw = torch.mm(do, v.t())
            ds = w * (dw - (w * dw).sum(1, keepdim=True)) * slant / D ** 0.5
            first = h % group == 0
            out["dq"][rq, cq] = torch.mm(ds, k)
            dk, dv = torch.mm(ds.t(), q), torch.mm(w.t(), do)
            out["dk"][rk, ck] = dk + (0 if first else out["dk"][rk, ck])
            out["dv"][rk, ck] = dv + (0 if first else out["dv"][rk, ck])
    return out
