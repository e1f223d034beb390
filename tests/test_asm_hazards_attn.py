"""Wait states before the attention kernels' inline-assembly LDS DMA instructions (host-only check of
the gfx950 assembly the compiler emits for csrc/attn_fwd.hip and csrc/attn_bwd.hip)."""

import os
import re
import subprocess

import pytest

from tests.test_asm_hazards import ROOT, _hipcc, dma_hazards


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")
@pytest.mark.parametrize("name", ["attn_fwd", "attn_bwd"])
def test_every_attention_dma_site_has_its_wait_states(name, tmp_path):
    out = tmp_path / f"{name}.s"
    src = os.path.join(ROOT, "fp8_blockwise_quantization_amd", "csrc", f"{name}.hip")
    cmd = [_hipcc(), "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"),
           "--cuda-device-only", "-S", "-o", str(out), src]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    text = out.read_text()
    assert len(re.findall(r"global_load_lds_dword", text)) > 50  # the DMA-fed kernels are in the file
    bad = dma_hazards(text)
    assert bad == [], f"{len(bad)} DMA sites lack wait states, e.g. {bad[:3]}"
