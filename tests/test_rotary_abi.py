"""Amplitudes that no float holds are refused before any CUDA call (no GPU needed)."""
import pytest

from bit_delta_tenant_gb300 import bitdelta as bd
from test_long_abi import A, lib  # noqa: F401


@pytest.mark.parametrize("amplitude,status", [(1e39, bd.BD_ERR_INVALID_ARG), (-1e300, bd.BD_ERR_INVALID_ARG), (3.4028235677973366e38, bd.BD_ERR_INVALID_ARG),
                                              (3.4028234e38, bd.BD_OK), (-3.4e38, bd.BD_OK), (0.0, bd.BD_OK), (1e-60, bd.BD_OK)])
def test_amplitudes(lib, amplitude, status):  # noqa: F811
    assert lib.bd_rotary_table(A, 0, 64, 1e4, 1.0, 0.0, 1.0, 4.0, amplitude, None) == status
