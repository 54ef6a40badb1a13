"""The experts' operators where their inputs are at an edge: rows that are not finite, rows that no pair has, panels of
scales, one workspace for many sizes; on the GPU against the fp64 oracle (oracle/experts.py)."""
import numpy as np
import pytest

from oracle import block, experts
from test_gpu_experts import TYPES, Case, Layer, check_tables, dev, guarded, host, log, paro, seed_of, within  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("E,k", [(3, 1), (8, 2), (64, 6), (65, 3), (300, 8)])
def test_route_gradient_of_rows_that_are_not_finite(paro, E, k, kind, normalize):
    """A NaN or +inf among the logits: softmax is NaN at every expert, and so is its gradient; normalised, the experts
    that are not taken have 0 whatever the others hold. Tokens without an expert, and the other rows, as ever."""
    rng = np.random.default_rng(E + k)
    M = 9
    x = rng.standard_normal((M, E))
    x[1, E // 2] = np.nan
    x[2, E - 1] = np.inf
    x[3] = -np.inf
    x[4, :E - 1], x[4, E - 1] = -np.inf, np.nan  # a token without an expert: no gradient
    x[5, 1:] = -np.inf
    x[6, 0], x[6, 1] = np.nan, np.inf
    x[7, E // 2:] = -np.inf
    x[7, 0] = np.nan
    xd = torch.from_numpy(x).to(TYPES[kind]).cuda()
    log(f"route gradient E={E} k={k} {kind} normalize={normalize}")
    r = paro.paro_experts_route(xd, k, normalize=normalize)
    dw = rng.standard_normal((M, k)).astype(np.float32)
    got = paro.paro_experts_route_backward(xd, r.ids, r.weights, dev(dw), normalize=normalize)
    torch.cuda.synchronize()
    got, ids = got.double().cpu().numpy(), host(r.ids)
    for m in (1, 2, 6, 7):
        taken = np.zeros(E, bool)
        taken[ids[m][ids[m] >= 0]] = True
        if not taken.any():
            assert not got[m].any(), m
        elif normalize:
            assert np.isnan(got[m][taken]).all() and not got[m][~taken].any(), m
        else:
            assert np.isnan(got[m]).all(), (m, got[m])
    assert (ids[3:5] == -1).all() and not got[3:5].any()
    fine = [0, 3, 5, 8]
    ref, err = experts.route_backward(xd.double().cpu().numpy()[fine], ids[fine], host(r.weights).astype(np.float64)[fine],
                                      dw.astype(np.float64)[fine], normalize)
    within(got[fine], ref, experts.stored(ref, err, kind), "dlogits")
