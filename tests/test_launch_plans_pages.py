"""Host-side check of the fork's sums (sv_pages.cuh), compiled with nvcc into a host
program; no GPU needed."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_56_gb300", "csrc")


def test_places_of_fresh_pages_fit_whatever_is_wanted(tmp_path):
    from speculative_decoding_verification_56_gb300 import build
    try:
        nvcc = build._nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    exe = tmp_path / "pages_plan_check"
    cmd = [nvcc, *build.ARCH_FLAGS, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", CSRC,
           os.path.join(ROOT, "tests", "pages_plan_check.cu"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:]
    assert "places checked" in r.stdout
