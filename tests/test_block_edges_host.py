"""Feed-forward products and AdamW on the CPU where arguments are at an edge: refused, or answered, before any GPU work."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def paro():
    import rotated_w4_linear_amd as p
    p.load_library()
    return p


D = ctypes.c_void_p(16 * 1024)
ODD = ctypes.c_void_p(16 * 1024 + 8)


def test_dz_without_activation_is_checked(paro):
    f = paro.load_library().paro_w4_linear_act_backward
    ws = ctypes.c_void_p(1 << 20)
    assert f(None, D, D, D, None, 0, D, ODD, D, 4, 64, 256, 128, ws, 1 << 30, None) == -5
    assert f(None, D, D, D, None, 0, D, ODD, None, 4, 64, 256, 128, None, 0, None) == -5
    assert f(None, D, D, D, None, 0, D, D, None, 4, 64, 256, 128, None, 0, None) == 0   # dz is dy: nothing to do
    assert f(None, D, D, D, None, 0, D, D, D, 4, 64, 256, 128, None, 0, None) == -7
