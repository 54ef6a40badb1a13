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


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("M,E,k,kind", [(1, 3, 2, "fp32"), (77, 64, 6, "bf16"), (300, 1000, 8, "fp16"), (9, 65, 65 % 16, "fp32")])
def test_route_gradient_in_place(paro, M, E, k, kind, normalize):
    """dlogits may be the logits."""
    rng = np.random.default_rng(M + E)
    x = base.logits_of(rng, M, E, kind).cuda()
    log(f"route gradient in place M={M} E={E} k={k} {kind} normalize={normalize}")
    r = paro.paro_experts_route(x, k, normalize=normalize)
    dw = dev(rng.standard_normal((M, k)).astype(np.float32))
    want = paro.paro_experts_route_backward(x, r.ids, r.weights, dw, normalize=normalize)
    got = paro.paro_experts_route_backward(x, r.ids, r.weights, dw, normalize=normalize, dlogits=x)
    bits = torch.int32 if x.element_size() == 4 else torch.int16
    torch.cuda.synchronize()
    assert got is x and torch.equal(got.view(bits), want.view(bits))


def test_route_captured_with_the_largest_tables(paro):
    """More LDS than a launch takes by itself, inside a capture; other logits at each replay."""
    M, E, k = 33000, 1024, 16
    x = torch.empty((M, E), device="cuda", dtype=torch.bfloat16)
    log("captured router")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = paro.paro_experts_route(x, k)
    for seed in range(3):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        g.replay()
        s = paro.paro_experts_route(x, k)
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(r, n), getattr(s, n)) for n in ("ids", "weights", "offsets", "order", "place"))


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


# ---------------------------------------------------------------------------
# what is not finite stays with its token
# ---------------------------------------------------------------------------

# every kernel of the products and of the gradients; numbers of weight rows that are no multiple of 64
ISOLATED = {"few rows": (3, 8, 2, 48, 1024, 128), "tiles of 16": (20, 8, 2, 272, 512, 128),
            "tiles of 32": (60, 6, 2, 272, 512, 64), "tiles of 48": (130, 4, 2, 528, 256, 128),
            "large tiles": (400, 2, 1, 272, 512, 128), "large tiles, panel": (700, 3, 1, 144, 1024, 64),
            "gradient shared out": (200, 4, 1, 1552, 4096, 128), "many experts": (600, 64, 2, 112, 1152, 64),
            "one expert": (260, 1, 1, 48, 256, 256)}


def spoilt(a, row, how):
    b = a.copy()
    if how == "mixed":
        b[row, ::3], b[row, 1::3] = np.nan, np.inf
    else:
        b[row, a.shape[1] // 2] = {"nan": np.nan, "inf": np.inf}[how]
    return b


@pytest.mark.parametrize("how", ["mixed", "nan", "inf"])
@pytest.mark.parametrize("name", list(ISOLATED))
def test_what_is_not_finite_stays_with_its_token(paro, name, how):
    """One token of X, one row of dH, one row of H, one token of dY, one weight: all that belongs to other tokens has the
    same bits as without it, and what belongs to this one is not finite."""
    M, E, k, N, d, G = ISOLATED[name]
    c = Case(paro, 31 + M, M, E, k, 2 * N, d, G, padded=0.05 if M > 100 else 0.0)
    pairs = c.order[:c.n]
    token = pairs // k
    x, dh = c.half(M, d), c.half(M * k, N)
    row = c.n // 2
    bad = token[row]
    others, rest = np.arange(M) != bad, token != bad
    bits = lambda t: host(t).view(np.int16 if t.element_size() == 2 else np.int32)  # noqa: E731
    spoils = lambda t: ~np.isfinite(host(t).astype(np.float32))  # noqa: E731

    def same(a, b, keep, what):
        assert np.array_equal(bits(a)[:len(keep)][keep], bits(b)[:len(keep)][keep]), f"{name} {how}: {what}"
    log(f"isolation {name} {how}: gated")
    gated = lambda x: paro.paro_w4_experts_gated(c.r, dev(x), *c.dev, bias=c.bd, group=G)  # noqa: E731
    back = lambda x, dh: paro.paro_w4_experts_gated_backward(c.r, dev(x), *c.dev, dev(dh), bias=c.bd, group=G)  # noqa: E731
    clean, worse = gated(x), gated(spoilt(x, bad, how))
    same(clean, worse, rest, "h")
    assert spoils(worse)[:c.n][~rest].any(1).all()
    log("  backward, X")
    (dx, dz), (dx1, dz1) = back(x, dh), back(spoilt(x, bad, how), dh)
    same(dz, dz1, rest, "dz")
    same(dx, dx1, others, "dx")
    assert spoils(dx1)[bad].any()
    log("  backward, dH")
    dx2, dz2 = back(x, spoilt(dh, row, how))
    same(dz, dz2, np.arange(c.n) != row, "dz")
    same(dx, dx2, others, "dx")
    assert spoils(dz2)[row].any() and spoils(dx2)[bad].all()
    c = Case(paro, 32 + M, M, E, k, N, d, G, padded=0.05 if M > 100 else 0.0)
    pairs = c.order[:c.n]
    token = pairs // k
    h, dy, res = c.half(M * k, d), c.half(M, N), c.half(M, N)
    row = c.n // 2
    bad = token[row]
    others, rest = np.arange(M) != bad, token != bad
    log("  combine")
    combine = lambda h: paro.paro_w4_experts_combine(c.r, dev(h), *c.dev, bias=c.bd, residual=dev(res), group=G)  # noqa: E731
    y, y1 = combine(h), combine(spoilt(h, row, how))
    same(y, y1, others, "y")
    assert spoils(y1)[bad].all()
    log("  backward, H")
    back = lambda h, dy: paro.paro_w4_experts_combine_backward(c.r, dev(h), *c.dev, dev(dy), bias=c.bd, group=G)  # noqa: E731
    (g, dw), (g1, dw1) = back(h, dy), back(spoilt(h, row, how), dy)
    same(g, g1, np.ones(c.n, bool), "dh")
    keep = np.arange(M * k) != pairs[row]
    same(dw.view(-1, 1), dw1.view(-1, 1), keep, "dweights")
    assert spoils(dw1).reshape(-1)[pairs[row]]
    log("  backward, dY")
    g2, dw2 = back(h, spoilt(dy, bad, how))
    same(g, g2, rest, "dh")
    same(dw, dw2, others, "dweights")
    assert spoils(g2)[:c.n][~rest].all() and spoils(dw2).reshape(-1)[pairs[~rest]].all()
    log("  a weight")
    c.r.weights.view(-1)[int(pairs[row])] = {"mixed": float("nan"), "nan": float("nan"), "inf": float("inf")}[how]
    y2, (g3, dw3) = combine(h), back(h, dy)
    same(y, y2, others, "y")
    same(g, g3, np.arange(c.n) != row, "dh")
    same(dw, dw3, np.ones(M, bool), "dweights")
    assert spoils(y2)[bad].all() and spoils(g3)[row].all()
