"""Feed-forward products and AdamW on the CPU where arguments are at an edge: refused, or answered, before any GPU work."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def test_backward_workspace_of_refused_sizes(paro):
    """Sizes that the calls refuse: no workspace, whatever they are, on both sides of 128 tokens."""
    import subprocess
    import sys
    # (in a process of its own: a division by zero ends it)
    code = """
import rotated_w4_linear_amd as p
lib = p.load_library()
for M in (1, 4, 128, 129, 1000, 1 << 40, (1 << 63) - 1):
    for N, d in ((64, 1), (64, 64), (64, 127), (64, 192), (17, 256), (8, 256), (1, 1), (1 << 22, 256), (64, 1 << 23)):
        for act in (0, 1):
            assert lib.paro_w4_linear_act_backward_workspace_size(M, N, d, act) == 0, (M, N, d)
        assert lib.paro_w4_gated_backward_workspace_size(M, N, d) == 0, (M, N, d)
for M in (1, 4, 128, 129):
    assert lib.paro_w4_linear_act_backward_workspace_size(M, 64, 128, 1) >= 16384
    assert lib.paro_w4_gated_backward_workspace_size(M, 64, 128) >= 16384
for M in (1 << 40, (1 << 63) - 1):
    assert lib.paro_w4_gated_backward_workspace_size(M, 64, 128) == 0
"""
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100, cwd=ROOT)
    assert res.returncode == 0, f"{res.returncode}: {res.stderr[-2000:]}"
    f = paro.load_library().paro_w4_linear_act_backward
    assert f(D, D, D, D, None, 1, D, D, D, 4, 64, 64, 64, None, 0, None) == -2
