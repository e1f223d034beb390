"""What the build needs for each of its parts (the compilers are stood in for: nothing is built)."""

import os

import pytest

from fp8_blockwise_quantization_amd import build as b


@pytest.fixture
def runs(monkeypatch, tmp_path):
    """The commands of a build into tmp_path, whose outputs are made empty."""
    seen = []

    def run(cmd, verbose):
        seen.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / b.LIB_NAME))
    monkeypatch.setattr(b, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))
    return seen


def test_the_library_alone_needs_no_host_compiler(runs, monkeypatch, tmp_path):
    monkeypatch.setattr(b, "cxx_path", lambda: pytest.fail("no host compiler is needed"))
    assert b.build(marshal=False) == str(tmp_path / b.LIB_NAME)
    assert len(runs) == 1 and os.listdir(tmp_path) == [b.LIB_NAME]


def test_both_parts_by_default(runs, tmp_path):
    b.build()
    assert len(runs) == 2 and sorted(os.listdir(tmp_path)) == ["_marshal.so", b.LIB_NAME]


def test_without_a_system_compiler_the_toolchains_own_is_taken(monkeypatch, tmp_path):
    for name in ("hipcc", "amdclang++"):
        (tmp_path / name).write_text("")
    monkeypatch.setattr(b.shutil, "which", lambda name: None)
    monkeypatch.setattr(b, "hipcc_path", lambda: str(tmp_path / "hipcc"))
    assert b.cxx_path() == str(tmp_path / "amdclang++")
    os.remove(tmp_path / "amdclang++")
    with pytest.raises(RuntimeError, match="C\\+\\+ compiler"):
        b.cxx_path()
