"""The host-side validation of include/fp8rl_attn.h under AddressSanitizer, as
tests/test_abi_block_asan.py does it for include/fp8rl_block.h. No kernel is launched.
"""

import os
import shutil
import subprocess
import sys

import pytest

from tests.test_abi_asan import ROOT, _asan_runtime


@pytest.mark.skipif(_asan_runtime() is None or shutil.which("hipcc") is None
                    and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="hipcc or the AddressSanitizer runtime is not available")
def test_attention_validation_under_address_sanitizer(tmp_path):
    from fp8_blockwise_quantization_amd import build as b

    lib = str(tmp_path / "libfp8rl_asan.so")
    b.build(extra_flags=["-Xarch_host", "-fsanitize=address", "-Xarch_host",
                         "-fno-omit-frame-pointer"], out_path=lib)
    env = dict(os.environ, LD_PRELOAD=_asan_runtime(), FP8RL_TEST_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               HIP_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-m", "pytest", "-v", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_attn_host.py"), "-k",
                        "not python_binding and not marshalling_module and not strict_c99"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "AddressSanitizer" not in out, out[-4000:]
    for name in ("decode_refusals", "decode_workspace", "read_refusals", "fwd_refusals", "bwd_refusals"):
        assert f"::test_{name} PASSED" in out, out[-4000:]
