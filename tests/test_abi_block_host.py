"""Host-side checks of include/fp8rl_block.h (CPU only: no kernel is ever launched here): the
library exports what the header declares, the header is strict C99 and its struct has the binding's
layout, and invalid arguments are refused with the documented status before any HIP call."""

import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

import fp8_blockwise_quantization_amd as fq
from fp8_blockwise_quantization_amd import _block, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8rl_block.h")

OK, ENULL, ESHAPE, EALIGN, EDTYPE, EWS, EHIP, EARG, ESCRATCH = range(9)
A = 1 << 20  # a fake, 16-byte aligned "device address": never dereferenced by these calls
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    other = os.environ.get("FP8RL_TEST_LIBRARY")
    return _block.declare_block(ctypes.CDLL(other) if other else _lib.lib())


def test_every_declared_symbol_is_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fp8rl_\w+)\s*\(", text)))
    assert sorted(_block.EXPORTED_BLOCK) == names
    for n in names:
        assert hasattr(L, n) and hasattr(fq, n), n


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_header_is_strict_c99_and_its_struct_is_the_bindings(tmp_path):
    src = tmp_path / "s.c"
    fields = [n for n, _ in _block.RopeKvArgs._fields_]
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"fp8rl_block.h\"\n"
                   "int main(void) {\n  printf(\"%zu\\n\", sizeof(fp8rl_rope_kv_args));\n"
                   + "".join(f"  printf(\"%zu\\n\", offsetof(fp8rl_rope_kv_args, {n}));\n"
                             for n in fields) + "  return 0;\n}\n")
    exe = tmp_path / "s"
    res = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                          os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(_block.RopeKvArgs)] + [getattr(_block.RopeKvArgs, n).offset
                                                        for n in fields]


def test_norm_refusals(L):
    base = dict(x=A, ldx=256, res=A, ldr=256, w=A, eps=1e-6, M=4, K=256, h=A, ldh=256, y=A, ldy=256,
                xq=A, ldq=256, sa=A, fmt=0)

    def call(**k):
        a = dict(base, **k)
        return L.fp8rl_add_rmsnorm_quant(*[a[n] for n in base], None)

    assert call(M=0, x=None) == OK
    assert call(K=0, ldx=0) == OK
    for n in ("x", "w"):
        assert call(**{n: None}) == ENULL, n
    assert call(xq=None) == ENULL  # codes without scales
    assert call(sa=None) == ENULL
    assert call(xq=None, sa=None, y=None) == ENULL  # nothing to write
    assert call(res=None) == EARG  # h without a residual
    for eps in (0.0, -1e-6, NAN, INF, 1e-39):
        assert call(eps=eps) == EARG, eps
    assert call(fmt=2) == EARG
    assert call(M=-1) == ESHAPE
    assert call(K=200) == ESHAPE
    assert call(K=32768 + 128, ldx=40000) == ESHAPE
    assert call(M=1 << 22) == ESHAPE
    for n in ("ldx", "ldr", "ldh", "ldy", "ldq"):
        assert call(**{n: 128}) == ESHAPE, n
        assert call(**{n: 260}) == EALIGN, n
    assert call(ldq=264) == EALIGN  # codes: a pitch that is a multiple of 16
    for n in ("x", "res", "w", "h", "y", "xq"):
        assert call(**{n: A + 8}) == EALIGN, n
    assert call(sa=A + 2) == EALIGN


def test_norm_bwd_refusals(L):
    base = dict(dy=A, ldy=256, h=A, ldh=256, w=A, dh=A, ldd=256, eps=1e-6, M=4, K=256, dx=A,
                ldx=256, dw=A, ws=A, wsb=1 << 30)

    def call(**k):
        a = dict(base, **k)
        return L.fp8rl_add_rmsnorm_bwd(*[a[n] for n in base], None)

    need = L.fp8rl_add_rmsnorm_bwd_workspace_bytes(4, 256)
    assert need > 0
    assert L.fp8rl_add_rmsnorm_bwd_workspace_bytes(-1, 256) == 0
    assert L.fp8rl_add_rmsnorm_bwd_workspace_bytes(4, 200) == 0
    assert call(M=0, dw=None, dy=None) == OK
    assert call(K=0) == OK
    for n in ("dy", "h", "w", "dx"):
        assert call(**{n: None}) == ENULL, n
    assert call(ws=None) == EWS
    assert call(wsb=need - 1) == EWS
    assert call(ws=A + 8) == EALIGN
    assert call(dw=A + 2) == EALIGN
    for eps in (0.0, NAN, INF):
        assert call(eps=eps) == EARG
    assert call(K=130) == ESHAPE
    assert call(M=-1) == ESHAPE
    for n in ("ldy", "ldh", "ldd", "ldx"):
        assert call(**{n: 128}) == ESHAPE, n
        assert call(**{n: 260}) == EALIGN, n
    for n in ("dy", "h", "w", "dh", "dx"):
        assert call(**{n: A + 8}) == EALIGN, n


def test_sort_refusals(L):
    base = dict(ids=A, kind=0, T=64, k=8, E=128, off=A, rows=A, pos=A, ws=A, wsb=1 << 30)

    def call(**k):
        a = dict(base, **k)
        return L.fp8rl_moe_sort(*[a[n] for n in base], None)

    for n in ("ids", "off", "rows", "pos"):
        assert call(**{n: None}) == ENULL, n
        assert call(**{n: A + 2}) == EALIGN, n
    assert call(kind=1, ids=A + 4) == EALIGN
    assert call(kind=2) == EDTYPE
    assert call(E=0) == EARG
    assert call(E=1025) == EARG
    assert call(k=0) == EARG
    assert call(k=65) == EARG
    assert call(T=-1) == ESHAPE
    assert call(T=1 << 24) == ESHAPE
    assert L.fp8rl_moe_sort_workspace_bytes(64, 8, 128) == 0
    need = L.fp8rl_moe_sort_workspace_bytes(65536, 8, 128)
    assert need > 0
    assert call(T=65536, ws=None) == EWS
    assert call(T=65536, wsb=need - 1) == EWS
    assert call(T=65536, ws=A + 4) == EALIGN
    assert call(T=0, off=None) == ENULL
    assert L.fp8rl_moe_sort_workspace_bytes(-1, 8, 128) == 0


def test_row_refusals(L):
    base = dict(x=A, ldx=64, pos=A, T=4, k=2, N=64, out=A, R=8, ldo=64)

    def call(**k):
        a = dict(base, **k)
        return L.fp8rl_moe_dispatch(*[a[n] for n in base], None)

    for n in ("T", "N", "R"):
        assert call(**{n: 0}, x=None) == OK, n
        assert call(**{n: -1}) == ESHAPE, n
    for n in ("x", "pos", "out"):
        assert call(**{n: None}) == ENULL, n
        assert call(**{n: A + 2}) == EALIGN, n
    assert call(N=60) == ESHAPE
    for n in ("ldx", "ldo"):
        assert call(**{n: 56}) == ESHAPE
        assert call(**{n: 68}) == EALIGN
    assert call(k=0) == EARG
    assert call(k=65) == EARG
    assert call(T=1 << 24) == ESHAPE
    assert call(T=1 << 20, N=1 << 17, ldx=1 << 17, ldo=1 << 17) == ESHAPE  # 2^26 waves

    base2 = dict(y=A, yt=0, R=8, ldy=64, pos=A, w=A, T=4, k=2, N=64, out=A, ot=0, ldo=64)

    def comb(**k):
        a = dict(base2, **k)
        return L.fp8rl_moe_combine(*[a[n] for n in base2], None)

    assert comb(T=0, y=None) == OK
    assert comb(N=0, y=None) == OK
    for n in ("y", "pos", "out"):
        assert comb(**{n: None}) == ENULL, n
    for n in ("y", "pos", "out", "w"):
        assert comb(**{n: A + 2}) == EALIGN, n
    assert comb(yt=2) == EDTYPE
    assert comb(ot=-1) == EDTYPE
    assert comb(ldy=56) == ESHAPE
    assert comb(ldo=68) == EALIGN
    assert comb(N=4) == ESHAPE
    assert comb(k=0) == EARG

    base3 = dict(g=A, ldg=64, y=A, ldy=64, yt=0, R=8, pos=A, w=A, T=4, k=2, N=64, dy=A, ldd=64, dw=A)

    def bwd(**k):
        a = dict(base3, **k)
        return L.fp8rl_moe_combine_bwd(*[a[n] for n in base3], None)

    assert bwd(T=0, g=None) == OK
    for n in ("g", "pos", "dy"):
        assert bwd(**{n: None}) == ENULL, n
    assert bwd(y=None) == ENULL  # dweights without y
    assert bwd(dw=None) == ENULL
    for n in ("g", "y", "pos", "w", "dy", "dw"):
        assert bwd(**{n: A + 2}) == EALIGN, n
    assert bwd(yt=5) == EDTYPE
    assert bwd(ldg=56) == ESHAPE
    assert bwd(ldd=68) == EALIGN


def test_append_refusals(L):
    base = dict(q=A, k=A, v=A, ld_q=512, ld_k=256, ld_v=256, T=4, q_heads=4, kv_heads=2,
                head_dim=128, rot_dim=128, interleaved=0, eps=1e-6, positions=A, cos_sin=A,
                max_pos=100, q_weight=A, k_weight=A, q_out=A, ld_qo=512, q_scale=None,
                slot_mapping=A, k_cache=A, v_cache=A, k_scale=A, v_scale=A, num_pages=4,
                page_size=16, page_stride=4096, slot_stride=256, head_stride=128)

    def call(**k):
        return L.fp8rl_rope_kv_append(ctypes.byref(_block.RopeKvArgs(**dict(base, **k))), None)

    assert L.fp8rl_rope_kv_append(None, None) == ENULL
    assert call(T=0, q=None, k=None) == OK
    for n in ("q", "k", "v", "q_out", "slot_mapping", "k_cache", "v_cache", "positions", "cos_sin",
              "q_weight", "k_scale"):
        assert call(**{n: None}) == ENULL, n
    for n in ("q", "k", "v", "q_out", "cos_sin", "q_weight", "k_weight"):
        assert call(**{n: A + 8}) == EALIGN, n
    for n in ("slot_mapping", "positions", "k_cache", "v_cache"):
        assert call(**{n: A + 4}) == EALIGN, n
    assert call(k_scale=None, v_scale=None, k_cache=A + 8) == EALIGN  # bf16 rows
    assert call(k_scale=A + 2) == EALIGN
    assert call(q_scale=A, q_out=A + 4) == EALIGN
    for n in ("ld_q", "ld_qo"):
        assert call(**{n: 504}) == ESHAPE, n
        assert call(**{n: 516}) == EALIGN, n
    for n in ("ld_k", "ld_v"):
        assert call(**{n: 248}) == ESHAPE, n
    for n in ("page_stride", "slot_stride", "head_stride"):
        assert call(**{n: 64}) == ESHAPE, n
        assert call(**{n: base[n] + 4}) == EALIGN, n
        assert call(**{n: 1 << 61}) == ESHAPE, n
    assert call(head_dim=120, rot_dim=128) == ESHAPE
    assert call(head_dim=4) == ESHAPE
    assert call(head_dim=520, rot_dim=0) == ESHAPE
    assert call(head_dim=100, rot_dim=0) == ESHAPE
    assert call(rot_dim=24) == ESHAPE
    assert call(rot_dim=-16) == ESHAPE
    assert call(kv_heads=0) == ESHAPE
    assert call(q_heads=-1) == ESHAPE
    assert call(T=-1) == ESHAPE
    assert call(T=1 << 26) == ESHAPE
    assert call(interleaved=2) == EARG
    assert call(eps=0.0) == EARG
    assert call(eps=NAN) == EARG
    assert call(page_size=0) == ESHAPE
    assert call(num_pages=-1) == ESHAPE
    assert call(num_pages=1 << 60) == ESHAPE
    assert call(max_pos=-1) == ESHAPE
    assert call(max_pos=1 << 31) == ESHAPE


def test_marshalling_module_refuses_before_any_launch():
    """The compiled checks by themselves: argument counts, types, tensors that are none or not on
    the device."""
    m = _block._marshal()
    x, w = torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros(128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        m.add_rmsnorm_quant(x, w)
    with pytest.raises(ValueError, match="x must be a device"):
        m.add_rmsnorm_quant(x, w, None, 1e-6, None, None, None, None, 0, 0, 0)
    with pytest.raises(ValueError, match="topk_ids must be a device"):
        m.moe_sort([1, 2], 4, None, None, None, None, 0, 0)
    with pytest.raises(TypeError):
        m.moe_combine(x, w, None, x, "0", 0)
    with pytest.raises(ValueError, match="k must be a device"):
        m.rope_kv_append(None, x, x, None, None, None, None, None, None, False, None, None, 1e-6,
                         None, None, None, 0, 0)


def test_python_binding_refuses_host_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        fq.add_rmsnorm_quant(bf(2, 128), bf(128))
    with pytest.raises(ValueError):
        fq.add_rmsnorm_bwd(bf(2, 128), bf(2, 128), bf(128))
    with pytest.raises(ValueError):
        fq.moe_sort(i32(2, 2), 4)
    with pytest.raises(ValueError):
        fq.moe_dispatch(bf(2, 128), i32(2, 2))
    with pytest.raises(ValueError):
        fq.moe_combine(y=bf(4, 128), pos=i32(2, 2))
    with pytest.raises(ValueError):
        fq.moe_combine_bwd(bf(2, 128), bf(4, 128), i32(2, 2))
    for q in (None, bf(2, 128)):
        with pytest.raises(ValueError):
            fq.rope_kv_append(q, bf(2, 128), bf(2, 128), None, None, None, bf(1, 16, 1, 128),
                              bf(1, 16, 1, 128))


@pytest.mark.parametrize("T,pieces", [(24573, 2731), (1082401, 62), (8191, 8193)])
def test_dispatch_refuses_a_grid_of_2_to_the_32_threads(L, T, pieces):
    """2^26 - 3 waves or more would round up to 2^24 workgroups of 256 threads, which HIP does not
    launch: refused by the documented bound, not by the launch."""
    assert (1 << 26) - 3 <= T * pieces < 1 << 26
    N = 2048 * pieces
    assert L.fp8rl_moe_dispatch(A, N, A, T, 1, N, A, 8, N, None) == ESHAPE


def test_a_marshalling_module_that_does_not_load_says_why(monkeypatch, tmp_path):
    """Built but not loadable (another torch's, say) is told apart from not built."""
    monkeypatch.setattr(_block, "_m", None)
    monkeypatch.delattr(fq, "_marshal", raising=False)
    monkeypatch.setitem(sys.modules, fq.__name__ + "._marshal", None)  # its import fails
    with pytest.raises(RuntimeError, match="cannot be loaded .*_marshal.*build it again") as e:
        _block._marshal()
    assert isinstance(e.value.__cause__, ImportError)
    monkeypatch.setattr(_block, "MARSHAL_PATH", str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match="is not built"):
        _block._marshal()


def test_sort_workspace_begins_past_one_workgroup(L):
    """4096 choices are one workgroup's, however they are shaped; 256 workgroups at most."""
    need = L.fp8rl_moe_sort_workspace_bytes
    for T, k in ((4096, 1), (512, 8), (64, 64), (585, 7), (0, 8)):
        assert need(T, k, 128) == 0, (T, k)
    for T, k, blocks in ((4097, 1, 2), (513, 8, 2), (65, 64, 2), (586, 7, 2), (1 << 20, 1, 256),
                         ((1 << 24) - 1, 64, 256)):
        assert need(T, k, 128) == blocks * 128 * 4, (T, k)
