"""The LDS that a launch sizes begins behind a kernel's own: where four floats at a time are stored there, on a 16-byte
boundary."""
import os
import re
import shutil
import subprocess

import pytest

from sharded_gemm_amd import build

SOURCES = ["linear_rows.hip"]      # those with LDS sized by the launch


def test_these_are_all():
    found = []
    for f in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, f)) as src:
            if "extern __shared__" in src.read():
                found.append(f)
    assert found == SOURCES


@pytest.mark.parametrize("src", SOURCES)
def test_launch_sized_lds_begins_aligned(src, tmp_path):
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("needs hipcc")
    out = str(tmp_path / "kernels.s")
    r = subprocess.run([build._hipcc(), *build.COMMON_FLAGS, "-x", "hip", "--offload-device-only", "-S",
                        os.path.join(build.CSRC, src), "-o", out], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    with open(out) as f:
        own = [int(v) for v in re.findall(r"^\s*\.group_segment_fixed_size:\s*(\d+)", f.read(), re.M)]
    assert own and all(n % 16 == 0 for n in own), own
