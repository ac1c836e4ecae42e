"""The decode step's operators through the bounds-checked build, in a child process (so that the debug library is the
one loaded); see test_gpu_debug_build.py."""
import os
import subprocess
import sys

import pytest

from bit_delta_tenant_gb300 import build as lib_build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_long_context_operators_pass_their_bounds_checks():
    lib_build.build(debug=True)
    res = subprocess.run([sys.executable, os.path.join(HERE, "debug_long_child.py")], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert "debug build ok" in res.stdout
