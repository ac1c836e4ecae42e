"""Every file that holds a kernel checks indices in the bounds-checked build (no GPU needed)."""
import glob
import os
import re

import pytest

from bit_delta_tenant_gb300 import build as lib_build

FILES = [f for f in sorted(glob.glob(os.path.join(lib_build.CSRC, "*.cu"))) if "__global__" in open(f).read()]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_kernels_check_their_indices(path):
    text = re.sub(r"//.*", "", open(path).read())
    assert len(re.findall(r"\bin_bounds\(", text)) >= 1
