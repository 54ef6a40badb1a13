"""The experts' operators where their inputs are at an edge: rows that are not finite, rows that no pair has, panels of
scales, one workspace for many sizes; on the GPU against the fp64 oracle (oracle/experts.py)."""
import numpy as np
import pytest

import test_gpu_experts as base
from oracle import experts
from test_gpu_experts import TYPES, Case, check_tables, dev, host, log, paro, seed_of, within  # noqa: F401

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


# ---------------------------------------------------------------------------
# the transform of the down projections' input, with tokens that have no expert
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("M,E,k,d,H,padded", [(600, 8, 2, 256, 512, 0.3), (900, 4, 2, 128, 768, 0.9), (600, 8, 2, 256, 512, 1.0),
                                              (700, 3, 1, 256, 1024, 0.1)])
def test_gradient_of_the_transform_between_the_products(paro, M, E, k, d, H, padded, given):
    """X through the experts' gated block, its rows transformed, the down projections on them, and back to the angles
    and scales of that transform: it sums over all rows, those that no pair has included. Memory that held NaN before."""
    import oracle
    import synthetic
    from oracle import metrics
    G = 128
    rng = np.random.default_rng(M + E)
    _, lay, _ = synthetic.linear_case(seed=5, M=1, d=H, N=16, group=G, K=4)
    rot = paro.Rotation(lay.pairs, lay.theta, lay.alpha, G)
    half = lambda *s: dev((rng.standard_normal(s) / np.sqrt(s[-1])).astype(np.float16))  # noqa: E731
    up = [t.view(E, 2 * H, -1) for t in paro.paro_quantize_weights(None, half(E * 2 * H, d), G)]
    down = [t.view(E, d, -1) for t in paro.paro_quantize_weights(rot, half(E * d, H), G)]
    x, dy = half(M, d) * 8, half(M, d)
    logits = rng.standard_normal((M, E)).astype(np.float32)
    logits[rng.random(M) < padded] = -np.inf
    r = paro.paro_experts_route(dev(logits), k)
    R = M * k
    log(f"transform between the products M={M} E={E} k={k} H={H} padded={padded} given={given}")
    torch.cuda.empty_cache()
    held = torch.full((1 << 26,), float("nan"), dtype=torch.float16, device="cuda")
    h = dh = None
    if given:  # a caller's own memory, zero-filled as the header says
        h, dh = (torch.full((R, H), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
        h.zero_()
        dh.zero_()
    del held
    h = paro.paro_w4_experts_gated(r, x, *up, h=h)
    hr = paro.paro_rotate(rot, h)
    y = paro.paro_w4_experts_combine(r, hr, *down)
    dh, dw = paro.paro_w4_experts_combine_backward(r, hr, *down, dy, dh=dh)
    gh, dth, dal = paro.paro_rotation_backward(rot, h, dh.float())
    torch.cuda.synchronize()
    n = int(host(r.offsets)[-1])
    assert torch.isfinite(y).all() and not host(h)[n:].any() and not host(dh)[n:].any() and not host(gh)[n:].any()
    want = oracle.rotation_backward(host(h)[:n], host(dh)[:n], lay.pairs, lay.theta, lay.alpha)
    metrics.assert_grad_close(host(gh)[:n], want[0], "gh")
    for got, ref, name in ((dth, want[1], "dtheta"), (dal, want[2], "dalpha")):
        if n == 0:
            assert not host(got).any()
        else:
            metrics.assert_grad_close(host(got), ref, name)


@pytest.mark.parametrize("E,k,N,d,tokens", [(2, 1, 128, 256, (1, 5, 31, 32, 33, 129, 319, 320, 321, 700)),
                                            (8, 2, 1040, 512, (1, 8, 9, 35, 36, 63, 64, 65, 100, 640, 641, 700)),
                                            (3, 2, 2064, 1152, (2, 24, 36, 37, 140, 240, 241, 400))])
def test_one_workspace_for_every_batch(paro, E, k, N, d, tokens):
    """The workspace of the largest number of tokens serves all of them, and nothing is written behind the room that a
    call's own sizes ask for; results as with a workspace that the call makes."""
    most = max(tokens)
    new = {"combine": paro.new_experts_combine_workspace, "gated_backward": paro.new_experts_gated_backward_workspace,
           "combine_backward": paro.new_experts_combine_backward_workspace}
    room = max([f(most, E, k, N, d).numel() for f in new.values()] +
               [t.numel() for t in [paro.new_experts_route_workspace(most, E, k)] if t is not None])
    ws = torch.empty(room, dtype=torch.uint8, device="cuda")
    g, c = Case(paro, 1, 1, E, k, 2 * N, d, 128), Case(paro, 2, 1, E, k, N, d, 128)
    rng = np.random.default_rng(E)
    half = lambda *s: dev(rng.standard_normal(s).astype(np.float16))  # noqa: E731

    def same(name, M, call):
        need = new[name](M, E, k, N, d).numel()
        ws.fill_(171)
        got, own = call(ws), call(None)
        torch.cuda.synchronize()
        assert (ws[need:] == 171).all(), (name, M)
        for a, b in zip(got, own):
            assert torch.equal(a, b), (name, M)
    for M in tokens:
        log(f"one workspace E={E} k={k} N={N} d={d} M={M}")
        logits = dev(rng.standard_normal((M, E)).astype(np.float32))
        r, s = paro.paro_experts_route(logits, k, workspace=ws), paro.paro_experts_route(logits, k)
        assert all(torch.equal(getattr(r, n), getattr(s, n)) for n in ("ids", "weights", "offsets", "order", "place"))
        x, h, dh, dy = half(M, d), half(M * k, d), half(M * k, N), half(M, N)
        same("combine", M, lambda w: (paro.paro_w4_experts_combine(r, h, *c.dev, bias=c.bd, workspace=w),))
        same("gated_backward", M, lambda w: paro.paro_w4_experts_gated_backward(r, x, *g.dev, dh, bias=g.bd, workspace=w))
        same("combine_backward", M,
             lambda w: paro.paro_w4_experts_combine_backward(r, h, *c.dev, dy, bias=c.bd, workspace=w))


@pytest.mark.parametrize("M,E,k", [((1 << 18) + 1, 60, 2), (1 << 20, 7, 1), ((1 << 20) + 77, 256, 2), (1 << 21, 1024, 1),
                                   ((1 << 20) - 1, 40, 16), ((1 << 24) - 1, 3, 1)])
def test_tables_of_very_many_tokens(paro, M, E, k):
    """Chunks of more tokens, up to the most pairs that a routing can have."""
    rng = np.random.default_rng(M % 1000 + E)
    log(f"tables M={M} E={E} k={k}")
    ids = rng.integers(-1, E, (M, k)).astype(np.int32)
    check_tables(paro.paro_experts_sort(dev(ids), E), ids)


# ---------------------------------------------------------------------------
# the large tiles with their panel of scales and zeros: a mean of 144 rows an expert and more, up to 64 groups along k,
# a multiple of 8
# ---------------------------------------------------------------------------

PANELS = [
    (400, 2, 1, 272, 1024, 128, 0.0), (700, 3, 1, 144, 512, 64, 0.0), (330, 2, 1, 80, 4096, 64, 0.0),
    (600, 2, 2, 272, 2048, 128, 0.0), (450, 3, 1, 528, 2048, 256, 0.0), (500, 4, 2, 16, 1536, 64, 0.05),
    (320, 2, 1, 1040, 8192, 128, 0.0), (200, 1, 1, 400, 1024, 64, 0.3), (900, 4, 2, 304, 4096, 256, 0.1),
    # (beside them: 72 groups, and 12, without a panel)
    (330, 2, 1, 80, 4608, 64, 0.0), (330, 2, 1, 80, 1536, 128, 0.0),
]


@pytest.mark.parametrize("M,E,k,N,d,G,padded", PANELS)
def test_gated_with_a_panel(paro, M, E, k, N, d, G, padded):
    base.test_gated(paro, M, E, k, N, d, G, padded)


@pytest.mark.parametrize("M,E,k,N,d,G,padded", PANELS)
def test_combine_with_a_panel(paro, M, E, k, N, d, G, padded):
    base.test_combine(paro, M, E, k, N, d, G, padded)


def test_panels_have_tiles_of_both_heights(paro):
    """An expert's rows in tiles of 256, its last up to 128 in ones of half the height: on panels of every group size."""
    seen = set()
    for M, E, k, N, d, G, padded in PANELS:
        assert M * k >= 144 * E and d >= 256
        if d // G % 8 == 0 and d // G <= 64:
            for seed in (0, 1):  # the two tests'
                c = Case(paro, seed_of(M, E, k, N, d, G, padded) + seed, M, E, k, (2 - seed) * N, d, G, padded)
                for n in np.diff(c.offsets):
                    rest = n % 256
                    seen |= {(G, seed, "whole")} if n >= 256 else set()
                    seen |= {(G, seed, "short" if rest <= 128 else "tall")} if rest else set()
    assert seen == {(G, s, h) for G in (64, 128, 256) for s in (0, 1) for h in ("whole", "short", "tall")}, sorted(seen)
