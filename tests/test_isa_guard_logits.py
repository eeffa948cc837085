"""The guards of test_isa_guard.py on the logits operators' sources: no
dynamic lane read of a spill reload, no call, no private memory."""

import os
import shutil
import subprocess

import pytest

from speculative_decoding_verification_sampling_amd import build as specv_build
from test_isa_guard import private_use, stale_lane_reads


@pytest.mark.parametrize("source,kernels", [("specv_adjust.hip", ("k_adjust", "k_history_add", "k_history_reset")),
                                            ("specv_record.hip", ("k_top_logits",)),
                                            ("specv_distill.hip", ("k_distill", "k_part_stats", "k_part_loss",
                                                                   "k_part_grad"))])
def test_guards(source, kernels, tmp_path):
    if shutil.which(specv_build.hipcc()) is None and not os.path.exists(specv_build.hipcc()):
        pytest.skip("hipcc not available")
    src = os.path.join(specv_build.CSRC, source)
    out = tmp_path / "kernels.s"
    flags = [f for f in specv_build.FLAGS if f not in ("-shared", "-fPIC")]
    r = subprocess.run([specv_build.hipcc(), *flags, "-I", specv_build.INCLUDE, "-I", specv_build.CSRC,
                        "--offload-device-only", "-S", src, "-o", str(out)],
                       capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0, r.stderr[-2000:]
    asm = out.read_text()
    assert all(k in asm for k in kernels)
    assert stale_lane_reads(asm) == []
    assert private_use(asm) == ([], 0)
