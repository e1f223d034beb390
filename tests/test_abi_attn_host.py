"""Host-side checks of include/fp8rl_attn.h (CPU only: no kernel is ever launched here): the library
exports what the header declares, the header is strict C99 and its structs have the binding's
layout, and invalid arguments are refused with the documented status before any HIP call."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from fp8_blockwise_quantization_amd import _attn, _block, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8rl_attn.h")
STRUCTS = {"fp8rl_attn_decode_args": _attn.AttnDecodeArgs, "fp8rl_kv_read_args": _attn.KvReadArgs,
           "fp8rl_attn_args": _attn.AttnArgs}

OK, ENULL, ESHAPE, EALIGN, EDTYPE, EWS, EHIP, EARG, ESCRATCH = range(9)
A = 1 << 20  # a fake, 16-byte aligned "device address": never dereferenced by these calls
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    other = os.environ.get("FP8RL_TEST_LIBRARY")
    return _attn.declare_attn(ctypes.CDLL(other) if other else _lib.lib())


def test_every_declared_symbol_is_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fp8rl_\w+)\s*\(", text)))
    assert sorted(_attn.EXPORTED_ATTN) == names
    for n in names:
        assert hasattr(L, n) and hasattr(fq, n), n


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
@pytest.mark.parametrize("name", STRUCTS)
def test_header_is_strict_c99_and_its_structs_are_the_bindings(tmp_path, name):
    src = tmp_path / "s.c"
    binding = STRUCTS[name]
    fields = [n for n, _ in binding._fields_]
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"fp8rl_attn.h\"\n"
                   f"int main(void) {{\n  printf(\"%zu\\n\", sizeof({name}));\n"
                   + "".join(f"  printf(\"%zu\\n\", offsetof({name}, {n}));\n" for n in fields)
                   + "  return 0;\n}\n")
    exe = tmp_path / "s"
    res = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                          os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(binding)] + [getattr(binding, n).offset for n in fields]


CACHE = dict(k_cache=A, v_cache=A, k_scale=A, v_scale=A, num_pages=4, page_size=16, page_stride=4096,
             slot_stride=256, head_stride=128, kv_heads=2, head_dim=128, page_table=A, ld_table=8,
             table_width=8)


def cache_refusals(call):
    for n in ("k_cache", "v_cache", "k_scale", "v_scale", "page_table"):
        assert call(**{n: None}) == ENULL, n
    for n in ("k_cache", "v_cache"):
        assert call(**{n: A + 4}) == EALIGN, n
    assert call(k_scale=None, v_scale=None, k_cache=A + 8) == EALIGN  # bf16 rows
    for n in ("k_scale", "page_table"):
        assert call(**{n: A + 2}) == EALIGN, n
    for n in ("page_stride", "slot_stride", "head_stride"):
        assert call(**{n: 64}) == ESHAPE, n
        assert call(**{n: CACHE[n] + 4}) == EALIGN, n
        assert call(**{n: 1 << 61}) == ESHAPE, n
    assert call(ld_table=7) == ESHAPE
    assert call(table_width=-1) == ESHAPE
    assert call(table_width=1 << 30) == ESHAPE  # 2^34 keys
    assert call(page_size=0) == ESHAPE
    assert call(num_pages=-1) == ESHAPE
    assert call(num_pages=1 << 60) == ESHAPE
    assert call(kv_heads=0) == ESHAPE


def test_decode_refusals(L):
    base = dict(CACHE, q=A, ld_q=1024, q_scale=None, B=4, q_heads=8, lengths=A, sm_scale=0.1,
                window=0, cap=0.0, slopes=A, out=A, ld_out=1024)

    def call(ws=A, wsb=1 << 40, **k):
        args = _attn.AttnDecodeArgs(**dict(base, **k))
        return L.fp8rl_attn_decode(ctypes.byref(args), ws, wsb, None)

    assert L.fp8rl_attn_decode(None, A, 0, None) == ENULL
    assert call(B=0, q=None, k_cache=None) == OK
    cache_refusals(call)
    for n in ("q", "lengths", "out"):
        assert call(**{n: None}) == ENULL, n
    for n in ("q", "out"):
        assert call(**{n: A + 8}) == EALIGN, n
    for n in ("q_scale", "lengths", "slopes"):
        assert call(**{n: A + 2}) == EALIGN, n
    assert call(q_scale=A, q=A + 4) == EALIGN
    for n in ("ld_q", "ld_out"):
        assert call(**{n: 1016}) == ESHAPE, n
        assert call(**{n: 1028}) == EALIGN, n
    for d in (0, 8, 40, 272):
        assert call(head_dim=d) == ESHAPE, d
    for h in (0, -8, 7, 9, 4098):
        assert call(q_heads=h) == ESHAPE, h
    assert call(B=-1) == ESHAPE
    assert call(B=65537) == ESHAPE
    assert call(B=65536, table_width=1 << 22, ld_table=1 << 22) == ESHAPE  # 2^42 keys in all
    assert call(B=65536, kv_heads=64, q_heads=64, ld_q=8192, ld_out=8192) == ESHAPE  # 2^22 pieces
    for v in (NAN, INF, -INF, 1e19):
        assert call(sm_scale=v) == EARG, v
    for v in (NAN, INF, -1.0, 1e-19, 1e19):
        assert call(cap=v) == EARG, v
    assert call(window=-1) == EARG


def test_decode_workspace(L):
    need = L.fp8rl_attn_decode_workspace_bytes
    assert need(4, 8, 2, 128, 1024, 0) == 0  # nothing is split up to there
    assert need(4, 8, 2, 256, 512, 0) == 0  # nor up to 256 KiB of a head's keys
    assert need(4, 8, 2, 256, 513, 0) > 0
    assert need(4, 8, 2, 128, 1 << 20, 200) == 0
    big = need(4, 8, 2, 128, 1025, 0)
    # two rows of four heads for each of 2048 waves, a word of every sequence and one of all
    assert big == 2 * 2048 * 4 * 130 * 4 + 5 * 4
    assert need(4, 8, 2, 128, 1 << 30, 0) == big  # bounded by the waves, not the length
    assert need(4, 8, 2, 128, 1 << 30, (1 << 31) - 1) == big
    assert need(0, 8, 2, 128, 1 << 30, 0) == 0
    for bad in ((-1, 8, 2, 128, 1025, 0), (4, 7, 2, 128, 1025, 0), (4, 8, 2, 120, 1025, 0),
                (4, 8, 2, 128, -1, 0), (4, 8, 2, 128, (1 << 30) + 1, 0), (4, 8, 2, 128, 1025, -1)):
        assert need(*bad) == 0, bad
    args = _attn.AttnDecodeArgs(**dict(CACHE, q=A, ld_q=1024, B=4, q_heads=8, lengths=A, sm_scale=0.1,
                                       out=A, ld_out=1024, table_width=128, ld_table=128))
    n = need(4, 8, 2, 128, 2048, 0)
    assert L.fp8rl_attn_decode(ctypes.byref(args), None, n, None) == EWS
    assert L.fp8rl_attn_decode(ctypes.byref(args), A, n - 1, None) == EWS
    assert L.fp8rl_attn_decode(ctypes.byref(args), A + 8, n, None) == EALIGN


def test_read_refusals(L):
    base = dict(CACHE, B=4, offsets=A, starts=A, R=100, k_out=A, v_out=A, ld_k=256, ld_v=256)

    def call(**k):
        return L.fp8rl_kv_read(ctypes.byref(_attn.KvReadArgs(**dict(base, **k))), None)

    assert L.fp8rl_kv_read(None, None) == ENULL
    assert call(R=0, k_out=None) == OK
    assert call(B=0, offsets=None) == OK
    assert call(num_pages=0, k_cache=None) == OK
    assert call(table_width=0, page_table=None) == OK
    cache_refusals(call)
    for n in ("offsets", "k_out", "v_out"):
        assert call(**{n: None}) == ENULL, n
    for n in ("k_out", "v_out"):
        assert call(**{n: A + 8}) == EALIGN, n
    for n in ("offsets", "starts"):
        assert call(**{n: A + 2}) == EALIGN, n
    for n in ("ld_k", "ld_v"):
        assert call(**{n: 248}) == ESHAPE, n
        assert call(**{n: 260}) == EALIGN, n
    for d in (0, 4, 100, 520):
        assert call(head_dim=d) == ESHAPE, d
    assert call(R=-1) == ESHAPE
    assert call(R=1 << 24) == ESHAPE
    assert call(B=1 << 20) == ESHAPE


DOCS = dict(q=A, k=A, v=A, ld_q=512, ld_k=256, ld_v=256, Tq=100, Tk=120, q_heads=4, kv_heads=2,
            head_dim=128, docs=3, q_offsets=A, k_offsets=A, causal=1, window=0, prefix=A, sm_scale=0.1,
            cap=0.0, slopes=A, out=A, ld_out=512, lse=A, dout=A, ld_dout=512, dq=A, dk=A, dv=A,
            ld_dq=512, ld_dk=256, ld_dv=256)


def attention_refusals(call, names, pitches, wide):
    for n in names:
        assert call(**{n: None}) == ENULL, n
    for n in names:
        if "offsets" not in n and n != "lse":
            assert call(**{n: A + 8}) == EALIGN, n
    for n in ("q_offsets", "k_offsets", "prefix", "slopes", "lse"):
        assert call(**{n: A + 2}) == EALIGN, n
    for n in pitches:
        assert call(**{n: DOCS[n] - 8}) == ESHAPE, n
        assert call(**{n: DOCS[n] + 4}) == EALIGN, n
        assert call(**{n: 1 << 24}) == ESHAPE, n
    for d in (0, 8, 40, wide):
        assert call(head_dim=d) == ESHAPE, d
    for h in (0, -4, 1, 3, 4098):
        assert call(q_heads=h) == ESHAPE, h
    assert call(kv_heads=0) == ESHAPE
    for n in ("Tq", "Tk", "docs"):
        assert call(**{n: -1}) == ESHAPE, n
        assert call(**{n: 1 << 24}) == ESHAPE, n
    assert call(docs=(1 << 20) - 1, q_heads=20, ld_q=2560, ld_out=2560,
                ld_dout=2560, ld_dq=2560) == ESHAPE  # 2^24 tiles
    assert call(causal=2) == EARG
    for v in (NAN, INF, 0.0, -1.0, 1e19):
        assert call(sm_scale=v) == EARG, v
    for v in (NAN, INF, -1.0, 1e-19, 1e19):
        assert call(cap=v) == EARG, v
    assert call(window=-1) == EARG


def test_fwd_refusals(L):
    def call(**k):
        return L.fp8rl_attn_fwd(ctypes.byref(_attn.AttnArgs(**dict(DOCS, **k))), None)

    assert L.fp8rl_attn_fwd(None, None) == ENULL
    assert call(Tq=0, q=None, out=None) == OK
    assert call(docs=0, q_offsets=None) == OK
    attention_refusals(call, ("q", "k", "v", "out", "q_offsets", "k_offsets"),
                       ("ld_q", "ld_k", "ld_v", "ld_out"), wide=272)


def test_bwd_refusals(L):
    need = L.fp8rl_attn_bwd_workspace_bytes(100, 120, 3, 4, 2, 128)
    assert need >= 2 * 100 * 4 * 4
    assert L.fp8rl_attn_bwd_workspace_bytes(1 << 20, 1 << 20, 1, 4, 2, 128) == 2 * (1 << 20) * 4 * 4
    for bad in ((-1, 120, 3, 4, 2, 128), (1 << 24, 120, 3, 4, 2, 128), (100, 120, 3, 0, 2, 128),
                (100, 120, 3, 4, 3, 128), (100, 120, 3, 4, 2, 136), (100, 120, -1, 4, 2, 128)):
        assert L.fp8rl_attn_bwd_workspace_bytes(*bad) == 0, bad

    def call(ws=A, wsb=1 << 40, **k):
        return L.fp8rl_attn_bwd(ctypes.byref(_attn.AttnArgs(**dict(DOCS, **k))), ws, wsb, None)

    assert L.fp8rl_attn_bwd(None, A, 0, None) == ENULL
    assert call(Tq=0, Tk=0, q=None, k=None) == OK
    assert call(docs=0, q_offsets=None) == OK
    attention_refusals(call, ("q", "k", "v", "out", "q_offsets", "k_offsets", "lse", "dout", "dq", "dk",
                              "dv"),
                       ("ld_q", "ld_k", "ld_v", "ld_out", "ld_dout", "ld_dq", "ld_dk", "ld_dv"),
                       wide=144)
    assert call(Tk=0, k=None, dk=None, dq=None) == ENULL
    assert call(Tq=0, q=None, dq=None, dv=None) == ENULL
    assert call(ws=None) == EWS
    assert call(wsb=need - 1) == EWS
    assert call(ws=A + 8) == EALIGN


def test_marshalling_module_refuses_before_any_launch():
    m = _block._marshal()
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        m.attn_decode(x)
    with pytest.raises(ValueError, match="q must be a device"):
        m.attn_decode(x, *[None] * 13, 0, 0)
    with pytest.raises(ValueError, match="page_table must be a device"):
        m.kv_read(*[x] * 9, 0, 0)
    with pytest.raises(ValueError, match="q must be a device"):
        m.attn_fwd(*[x] * 14, 0, 0)
    with pytest.raises(ValueError, match="q must be a device"):
        m.attn_bwd(*[x] * 19, 0, 0)


def test_python_binding_refuses_host_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    cache = bf(2, 16, 1, 64)
    with pytest.raises(ValueError):
        fq.attn_decode(bf(2, 64), cache, cache, i32(2, 1), i32(2))
    with pytest.raises(ValueError):
        fq.kv_read(cache, cache, i32(2, 1), i32(3), rows=4)
    with pytest.raises(ValueError):
        fq.attn_fwd(bf(2, 64), bf(2, 64), bf(2, 64), 64, i32(2))
    with pytest.raises(ValueError):
        fq.attn_bwd(*[bf(2, 64)] * 5, torch.zeros(1, 2), 64, i32(2))
