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


# ---------------------------------------------------------------------------
# a workspace for the largest batch serves the smaller ones
# ---------------------------------------------------------------------------

def sizes_up_to(size, M, *rest):
    return [size(m, *rest) for m in M]


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (256, 8), (1024, 16), (1000, 1)])
def test_route_workspace_never_shrinks(paro, E, k):
    size = paro.load_library().paro_experts_route_workspace_size
    edges = [128, 129, 16384, 32768, 65536, 1 << 17, 1 << 18, 1 << 19, 1 << 20, 1 << 21, 1 << 22, 1 << 23]
    M = sorted({m + i for m in edges for i in range(-260, 261)} | set(range(1, 4000)) | set(range(4000, 300000, 997)))
    M = [m for m in M if 0 < m < (1 << 24) // k]
    got = sizes_up_to(size, M, E, k)
    assert all(a <= b for a, b in zip(got, got[1:]))
    assert got[0] == 0 and got[-1] > 0


@pytest.mark.parametrize("E,k,N,d", [(8, 2, 4096, 14336), (8, 2, 14336, 4096), (64, 8, 1024, 2048), (32, 4, 1536, 2048),
                                     (60, 4, 2064, 1408), (128, 8, 512, 1024), (1, 1, 16, 128), (1, 1, 4096, 4096),
                                     (2, 2, 8192, 128), (3, 1, 2064, 256), (1024, 16, 64, 128), (256, 8, 32, 7168),
                                     (7, 3, 48, 384), (16, 1, 20000, 640)])
def test_product_workspaces_never_shrink(paro, E, k, N, d):
    for call in ("gated", "combine", "gated_backward", "combine_backward"):
        size = getattr(paro.load_library(), f"paro_w4_experts_{call}_workspace_size")
        M = list(range(1, 6000)) + list(range(6000, 60000, 61))
        M = [m for m in M if m * k < 1 << 24 and m * k * max(2 * N, d) < 1 << 34]
        got = sizes_up_to(size, M, E, k, N, d)
        shrinks = [(m, a, b) for m, a, b in zip(M[1:], got, got[1:]) if a > b]
        assert not shrinks, (call, shrinks[:5])
        if call != "gated":
            assert got[0] > 0
