"""Static checks of the attention tiles' generated code (no GPU needed): the copies into
LDS are inline asm, so the wait states that the compiler does not see are checked on its
output, as for the retrieval kernels, and the kernels must not spill."""
from __future__ import annotations

import subprocess

import pytest

from cross_model_sparse_amd import build, isa_check


@pytest.fixture(scope="module")
def findings(tmp_path_factory):
    if not isa_check.Path(build.HIPCC).exists():
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa") / "k_attn.s"
    cmd = [build.HIPCC, *build.DEVICE_FLAGS, *build.EXTRA_FLAGS["k_attn.hip"], "--cuda-device-only", "-S",
           str(build.CSRC / "k_attn.hip"), "-o", str(out)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    return isa_check.check_asm(str(out), pattern="k_attn")


def test_attention_kernels_have_no_hazards_and_do_not_spill(findings):
    tiles = {n: r for n, r in findings.items() if "k_attn_tiles" in n}
    assert len(tiles) == 6 and len(findings) == 18
    for name, r in findings.items():
        assert r["scratch"] == 0, name
        assert not r["valu_sgpr"], (name, r["valu_sgpr"][:3])
        assert not r["m0_dma"], (name, r["m0_dma"][:3])
        assert not r["m0_live"], (name, r["m0_live"][:3])
