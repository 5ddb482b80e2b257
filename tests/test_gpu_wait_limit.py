"""How long the waits between the roles of the tree attention over 4-bit pages last
when nobody answers: the limit that was set, by the GPU's clock.  The waits run in a
kernel of the test's own, on a barrier that nothing completes, and end by themselves."""
import os
import subprocess

import pytest

from speculative_decoding_verification_56_gb300 import build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MORE_NS = 5_000_000


def test_waits_that_run_out_keep_their_limit(tmp_path):
    """No sooner than the limit (the clock's steps of up to a microsecond aside), and
    not much later: one test before the first look at the clock and one that begins
    right before the end, each an eighth of the limit or a few microseconds."""
    exe = tmp_path / "wait_limit_check"
    subprocess.run([build._nvcc(), *build.ARCH_FLAGS, "-std=c++17", "-O3", "-I", build.INCLUDE, "-I", build.CSRC,
                    os.path.join(ROOT, "tests", "wait_limit_check.cu"), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    lines = [tuple(int(x) for x in line.split()) for line in r.stdout.splitlines()]
    assert len(lines) == 7 * 7
    for warp, kind, limit, took, ok in lines:
        what = (warp, kind, limit, took)
        late = limit // 4 + 100_000
        if kind == 0:    # nobody answers
            assert not ok and limit - 1000 <= took + (limit <= 1) <= limit + late, what
        elif kind == 1:  # another role has given up
            assert not ok and took <= late, what
        elif kind == 2:  # the phase is complete
            assert ok and took <= 20_000, what
        else:
            assert not ok and limit + MORE_NS - 1000 <= took <= limit + MORE_NS + late, what
