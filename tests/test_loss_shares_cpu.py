"""How the loss's second product shares its tiles among workgroups, checked on the host (tests/cpu/loss_shares.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_every_step_is_shared_out_once(tmp_path):
    exe = str(tmp_path / "loss_shares")
    r = subprocess.run([HIPCC, "-std=c++17", "-O2", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                        "-Wno-unused-command-line-argument", "-I", os.path.join(ROOT, "bit_nf4_quantized_codebook_amd", "csrc"),
                        "-x", "hip", os.path.join(ROOT, "tests", "cpu", "loss_shares.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
