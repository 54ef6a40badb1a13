"""The experts' operators on the CPU where their arguments are at an edge: what their calls make, and the workspaces
that they ask for."""
import pytest


@pytest.fixture(scope="module")
def paro():
    import rotated_w4_linear_amd as p
    p.load_library()
    return p


def test_rows_by_expert_that_a_call_makes_hold_no_garbage(paro, monkeypatch):
    """h and dh go through the transform and its gradient whole: rows that no pair has are 0 where the call made them."""
    import torch

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("size") else 0

    class Routing:
        M, E, k = 6, 4, 2

        def _on(self, device):
            return None
    monkeypatch.setattr(paro, "load_library", Lib)
    monkeypatch.setattr(paro, "_expect", lambda *a: 0)
    monkeypatch.setattr(paro, "_raw_stream", lambda *a: 0)
    monkeypatch.setattr(paro, "_workspace", lambda *a: (None, None, 0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    half = lambda *s: torch.ones(s, dtype=torch.float16)  # noqa: E731
    w = [torch.zeros(4, 64, n) for n in (128, 2, 2)]
    held = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)  # (memory that is not filled holds NaN)
    try:
        assert torch.isnan(torch.empty(3)).all()
        h = paro.paro_w4_experts_gated(Routing(), half(6, 256), *w)
        dh, _ = paro.paro_w4_experts_combine_backward(Routing(), half(12, 256), *w, half(6, 64))
    finally:
        torch.use_deterministic_algorithms(held)
    assert h.shape == (12, 32) and h.dtype == torch.float16 and not h.any()
    assert dh.shape == (12, 256) and dh.dtype == torch.float16 and not dh.any()
