"""A window that 32 bits do not hold: the largest one that they do stands for it, and a negative one stays negative."""
import pytest

from bit_delta_tenant_gb300 import bitdelta as bd
from test_binding_device import lib, step_calls  # noqa: F401


@pytest.mark.parametrize("window,given", [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                          (-1, -1), (-2 ** 32 + 5, -1)])
def test_window(lib, monkeypatch, window, given):  # noqa: F811
    seen = []
    monkeypatch.setattr(lib, "bd_attention_decode", lambda *args: seen.append(args) or 0, raising=False)
    call, tensors, plain = step_calls()[4]
    call(**tensors, **plain, window=window, stream=5)
    assert seen[0][8] == given
