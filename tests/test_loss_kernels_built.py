"""The library holds no kernel of the weight gradient's that no call can launch."""
import os
import re
import shutil
import subprocess

import pytest

from sharded_gemm_amd import _abi


def test_the_weight_gradient_has_no_32_deep_tile():
    """Its sum runs over tokens in multiples of 64."""
    if not os.path.exists(_abi.LIB_PATH) or shutil.which("nm") is None:
        pytest.skip("needs the built library and nm")
    names = subprocess.run(["nm", "-C", _abi.LIB_PATH], capture_output=True, text=True, check=True).stdout
    tiles = set(re.findall(r"lin_ring_kernel<(\d+), (\d+), (\d+), \d+, 7, true, true,", names))
    assert ("128", "128", "32") in tiles and ("64", "64", "64") in tiles
    assert ("64", "64", "32") not in tiles
