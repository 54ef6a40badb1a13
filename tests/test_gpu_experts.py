"""The experts' operators on the GPU against the fp64 oracle, value by value, within the
bounds that follow from the documented arithmetic (oracle/experts.py)."""
import numpy as np
import pytest

from oracle import block, experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def paro():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rotated_w4_linear_amd as p
    p.load_library()
    p.paro_device_init()
    return p


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def log(msg):
    print(msg, flush=True)


def within(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, what
    same_nan = np.isnan(ref) & np.isnan(got)
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - ref) <= tol) | same_nan | (got == ref))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} against {ref[bad][0]}, bound {np.broadcast_to(tol, ref.shape)[bad][0]}")


TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# the router
# ---------------------------------------------------------------------------

ROUTES = [(1, 1, 1), (1, 128, 8), (3, 2, 2), (7, 8, 2), (63, 65, 3), (64, 64, 16), (65, 64, 6), (300, 1000, 8),
          (1000, 8, 2), (777, 129, 5), (5000, 256, 8), (130, 1024, 16), (128, 1024, 16), (129, 100, 2), (256, 1024, 16), (257, 100, 2), (600, 1024, 16), (70000, 7, 2), (20000, 30, 3), (70, 3, 3), (2000, 200, 7),
          (33000, 1024, 16)]


def logits_of(rng, M, E, kind):
    x = rng.standard_normal((M, E)) * 2
    x[rng.random((M, E)) < 0.05] = -np.inf
    x = torch.from_numpy(x).to(TYPES[kind])
    if E > 3:
        x[:, 2] = x[:, 1]  # ties
        x[::2, 0], x[::2, 3] = 0.0, -0.0
    x[M // 2] = -np.inf  # a token whose mask leaves nothing
    if M > 4:
        x[M // 3, 1:] = -np.inf  # and one that has a single expert
        x[M // 4, E // 2] = float("nan")
    return x


def check_tables(r, ids):
    offsets, order, place = experts.tables(ids, r.E)
    assert np.array_equal(host(r.offsets), offsets)
    assert np.array_equal(host(r.order), order)
    assert np.array_equal(host(r.place), place)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,E,k", ROUTES)
def test_route(paro, M, E, k, kind):
    rng = np.random.default_rng(M * 7 + E + k)
    x = logits_of(rng, M, E, kind)
    xd = x.cuda()
    for normalize in (True, False):
        log(f"route M={M} E={E} k={k} {kind} normalize={normalize}")
        r = paro.paro_experts_route(xd, k, normalize=normalize)
        ids, w = experts.route(x.double().numpy(), k, normalize)
        assert np.array_equal(host(r.ids), ids)
        within(host(r.weights), w, experts.route_tolerance(x.double().numpy(), ids, w, normalize), "weights")
        check_tables(r, ids)
        # the tables alone, from the ids
        s = paro.paro_experts_sort(r.ids, E)
        for a, b in ((r.offsets, s.offsets), (r.order, s.order), (r.place, s.place)):
            assert torch.equal(a, b)
        dw = rng.standard_normal((M, k)).astype(np.float32)
        got = paro.paro_experts_route_backward(xd, r.ids, r.weights, dev(dw), normalize=normalize)
        torch.cuda.synchronize()
        keep = ~torch.isnan(x.double()).any(1).numpy()  # (a NaN's row: NaN weights)
        ref, err = experts.route_backward(x.double().numpy()[keep], ids[keep], host(r.weights).astype(np.float64)[keep],
                                          dw.astype(np.float64)[keep], normalize)
        within(got.double().cpu().numpy()[keep], ref, experts.stored(ref, err, kind), "dlogits")


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (40, 7, 3), (64, 1024, 16), (100, 3, 1), (2000, 60, 4), (4097, 500, 2)])
def test_sort_of_any_ids(paro, M, E, k):
    """Ids of another router: some of no expert, an expert twice for a token, all pairs of one expert, or none."""
    rng = np.random.default_rng(M + E)
    for case in ("any", "one", "none"):
        ids = rng.integers(-3, E + 3, (M, k)) if case == "any" else np.full((M, k), E - 1 if case == "one" else -1)
        log(f"sort M={M} E={E} k={k} {case}")
        check_tables(paro.paro_experts_sort(dev(ids.astype(np.int32)), E), ids)


def test_route_of_infinite_logits(paro):
    """+inf is taken first; its weights are NaN, as its softmax is, and the other rows are not touched."""
    x = torch.zeros((3, 8), device="cuda")
    x[1, 5] = float("inf")
    r = paro.paro_experts_route(x, 2)
    assert host(r.ids).tolist() == [[0, 1], [5, 0], [0, 1]]
    assert torch.isnan(r.weights[1]).any() and torch.equal(r.weights[::2], torch.full((2, 2), 0.5, device="cuda"))


# ---------------------------------------------------------------------------
# the products
# ---------------------------------------------------------------------------

class Case:
    """Random codes, scales, zeros and biases of E experts, and a routing."""

    def __init__(self, paro, seed, M, E, k, P, d, group, padded=0.0, skew=1.0, bias=True):
        rng = np.random.default_rng(seed)
        self.rng, self.M, self.E, self.k, self.P, self.d, self.group = rng, M, E, k, P, d, group
        self.qw = rng.integers(0, 256, (E, P, d // 2), dtype=np.uint8)
        self.s = (rng.uniform(0.5, 1.5, (E, P, d // group)) * 0.5 / np.sqrt(d)).astype(np.float16)
        self.z = rng.integers(5, 11, (E, P, d // group)).astype(np.uint8)
        self.b = (rng.standard_normal((E, P)) * 0.3).astype(np.float16) if bias else None
        x = rng.standard_normal((M, E)) + skew * rng.standard_normal((1, E))
        x[rng.random(M) < padded] = -np.inf
        self.r = paro.paro_experts_route(dev(x.astype(np.float32)), k)
        self.offsets, self.order, self.place = (host(t) for t in (self.r.offsets, self.r.order, self.r.place))
        self.weights = host(self.r.weights)
        self.n = int(self.offsets[-1])
        self.dev = [dev(a) for a in (self.qw, self.s, self.z)]
        self.bd = dev(self.b)

    def half(self, *shape):
        return self.rng.standard_normal(shape).astype(np.float16)

    def w(self):
        return [block.weights(self.qw[e], self.s[e], self.z[e], self.group) for e in range(self.E)]


def guarded(rows, cols, n, fill=777.0, dtype=None):
    """[rows][cols] output inside a larger buffer; its rows from n on, and the buffer around it, must stay as they are."""
    buf = torch.full(((rows + 16) * cols,), fill, dtype=dtype or torch.float16, device="cuda")
    out = buf[8 * cols:(rows + 8) * cols].view(rows, cols)

    def check():
        torch.cuda.synchronize()
        assert (buf[:8 * cols] == fill).all() and (buf[(n + 8) * cols:] == fill).all(), "written outside the output"
    return out, check


# M, E, k, N, d, group, padded: one token to many, experts without rows, one expert for
# all, every expert for all, odd numbers of everything, groups of 64, 128 and 256
PRODUCTS = [
    (1, 1, 1, 16, 128, 128, 0.0), (1, 8, 2, 48, 256, 128, 0.0), (1, 4, 4, 1040, 512, 64, 0.0),
    (1, 8, 2, 256, 4096, 128, 0.0), (1, 2, 2, 4112, 640, 128, 0.0), (2, 16, 8, 64, 1024, 256, 0.0),
    (3, 5, 3, 80, 384, 64, 0.0), (4, 8, 2, 512, 2048, 128, 0.3), (5, 1, 1, 272, 768, 256, 0.0),
    (16, 8, 2, 144, 1536, 128, 0.0), (16, 4, 1, 2064, 640, 64, 0.2), (17, 64, 8, 32, 256, 128, 0.0),
    (33, 3, 2, 528, 512, 128, 0.0), (64, 64, 8, 64, 512, 64, 0.1), (100, 8, 2, 208, 2560, 128, 0.0),
    (130, 100, 4, 48, 384, 128, 0.5), (200, 2, 1, 1040, 1024, 64, 0.0), (333, 16, 3, 336, 896, 128, 0.1),
    (700, 4, 2, 272, 512, 256, 0.0), (1500, 8, 2, 288, 256, 64, 0.05), (2500, 3, 1, 528, 384, 128, 0.0),
    (300, 2, 2, 64, 128, 128, 0.0), (400, 3, 1, 80, 256, 64, 0.2), (260, 1, 1, 48, 256, 256, 0.0),
    (150, 2, 2, 160, 640, 128, 0.0), (1200, 40, 6, 96, 384, 128, 0.0),
    (40, 64, 4, 1040, 640, 64, 0.0), (64, 48, 8, 816, 256, 256, 0.1), (130, 100, 4, 400, 384, 128, 0.5),
    (500, 40, 2, 880, 896, 64, 0.0), (150, 50, 4, 784, 128, 128, 0.0), (300, 30, 4, 1296, 1152, 128, 0.05),
    (90, 40, 8, 1056, 768, 256, 0.0), (33, 70, 7, 528, 1408, 64, 0.0), (20, 36, 6, 1040, 1280, 256, 0.0),
    (700, 100, 4, 80, 768, 128, 0.2), (600, 64, 2, 112, 1152, 64, 0.1),
    # (the gated gradient's tiles shared out: 2, 3 and 4 ways, the last range not whole k-tiles)
    (200, 4, 1, 1552, 4096, 128, 0.0), (150, 8, 2, 1600, 2304, 64, 0.1), (140, 3, 2, 2064, 1152, 128, 0.0),
    # no token has an expert
    (1, 8, 2, 48, 256, 128, 1.0), (5, 70, 3, 528, 384, 64, 1.0), (700, 4, 2, 272, 512, 256, 1.0),
]


def seed_of(*v):
    return sum(int(a * 10) * p for a, p in zip(v, (1, 31, 1009, 7, 5, 3, 11)))


@pytest.mark.parametrize("M,E,k,N,d,G,padded", PRODUCTS)
def test_gated(paro, M, E, k, N, d, G, padded):
    c = Case(paro, seed_of(M, E, k, N, d, G, padded), M, E, k, 2 * N, d, G, padded)
    w, x = c.w(), c.half(M, d)
    dh = c.half(M * k, N)
    ws = paro.new_experts_gated_workspace(M, E, k, N, d)
    wb = paro.new_experts_gated_backward_workspace(M, E, k, N, d)
    for i, name in enumerate(("silu", "gelu", "gelu_tanh", "relu", "none")[:2 if M > 300 else 5]):
        bias, bd = (c.b, c.bd) if i % 2 == 0 else (None, None)
        log(f"experts gated M={M} E={E} k={k} N={N} d={d} G={G} padded={padded} {name} bias={bias is not None}")
        h, check = guarded(M * k, N, c.n)
        paro.paro_w4_experts_gated(c.r, dev(x), *c.dev, bias=bd, act=name, h=h, group=G, workspace=ws)
        check()
        ref, tol = experts.gated(c.offsets, c.order, k, x, w, bias, name)
        within(host(h)[:c.n], ref[:c.n], tol[:c.n], f"{name} h")
        log("  backward")
        dz, check = guarded(M * k, 2 * N, c.n)
        dx, check_x = guarded(M, d, M)
        paro.paro_w4_experts_gated_backward(c.r, dev(x), *c.dev, dev(dh), bias=bd, act=name, dz=dz, dx=dx, group=G,
                                            workspace=wb)
        check()
        check_x()
        ref, tol = experts.gated_backward_dz(c.offsets, c.order, k, x, w, bias, name, dh)
        within(host(dz)[:c.n], ref[:c.n], tol[:c.n], f"{name} dz")
        ref, tol = experts.gated_backward_dx(c.offsets, c.order, k, M, w, host(dz))
        within(host(dx), ref, tol, f"{name} dx")
    # dz alone, without a workspace
    only, again = paro.paro_w4_experts_gated_backward(c.r, dev(x), *c.dev, dev(dh), bias=bd, act=name, want_dx=False,
                                                      group=G)
    assert only is None and torch.equal(again[:c.n], dz[:c.n])


@pytest.mark.parametrize("M,E,k,N,d,G,padded", PRODUCTS)
def test_combine(paro, M, E, k, N, d, G, padded):
    c = Case(paro, seed_of(M, E, k, N, d, G, padded) + 1, M, E, k, N, d, G, padded)
    w, h = c.w(), c.half(M * k, d)
    h[c.n:] = np.nan  # rows that no pair has are not read
    res, dy = c.half(M, N), c.half(M, N)
    ws = paro.new_experts_combine_workspace(M, E, k, N, d)
    wb = paro.new_experts_combine_backward_workspace(M, E, k, N, d)
    for bias, bd, residual in [(c.b, c.bd, res), (None, None, None)]:
        log(f"experts combine M={M} E={E} k={k} N={N} d={d} G={G} padded={padded} bias={bias is not None}")
        y, check = guarded(M, N, M)
        paro.paro_w4_experts_combine(c.r, dev(h), *c.dev, bias=bd, residual=dev(residual), y=y, group=G, workspace=ws)
        check()
        within(host(y), *experts.combine(c.offsets, c.order, k, h, w, bias, c.weights, residual), "y")
        log("  backward")
        dh, check = guarded(M * k, d, c.n)
        dw, check_w = guarded(M, k, M, dtype=torch.float32)
        paro.paro_w4_experts_combine_backward(c.r, dev(h), *c.dev, dev(dy), bias=bd, dh=dh, dweights=dw.contiguous(),
                                              group=G, workspace=wb)
        check()
        check_w()
        ref = experts.combine_backward(c.offsets, c.order, k, h, w, bias, c.weights, dy)
        within(host(dh)[:c.n], ref[0][:c.n], ref[1][:c.n], "dh")
        within(host(dw), ref[2], ref[3], "dweights")
    # the residual replaced in place
    y = dev(res)
    paro.paro_w4_experts_combine(c.r, dev(h), *c.dev, residual=y, y=y, group=G, workspace=ws)
    assert torch.equal(y, paro.paro_w4_experts_combine(c.r, dev(h), *c.dev, residual=dev(res), group=G))


def test_a_row_stays_by_itself(paro):
    """A token that is not finite spoils its own rows only, in every direction; a weight that is NaN its own token."""
    M, E, k, N, d, G = 90, 6, 2, 272, 512, 128
    c = Case(paro, 4, M, E, k, 2 * N, d, G)
    x, dh = c.half(M, d), c.half(M * k, N)
    bad = x.copy()
    bad[41, ::3], bad[41, 1::3] = np.nan, np.inf
    token = c.order[:c.n] // k
    mine = token == 41
    log("gated with a token that is not finite")
    a = [host(paro.paro_w4_experts_gated(c.r, dev(v), *c.dev, group=G))[:c.n] for v in (x, bad)]
    assert np.array_equal(a[0][~mine], a[1][~mine]) and not np.isfinite(a[1][mine]).any()
    b = [paro.paro_w4_experts_gated_backward(c.r, dev(v), *c.dev, dev(dh), group=G) for v in (x, bad)]
    assert np.array_equal(host(b[0][1])[:c.n][~mine], host(b[1][1])[:c.n][~mine])
    keep = np.arange(M) != 41
    assert np.array_equal(host(b[0][0])[keep], host(b[1][0])[keep])
    log("combine with a weight that is not finite")
    c = Case(paro, 5, M, E, k, N, d, G)
    h, dy = c.half(M * k, d), c.half(M, N)
    y = host(paro.paro_w4_experts_combine(c.r, dev(h), *c.dev, group=G))
    c.r.weights[41, 0] = float("nan")
    z = host(paro.paro_w4_experts_combine(c.r, dev(h), *c.dev, group=G))
    assert np.array_equal(y[keep], z[keep]) and np.isnan(z[41]).all()


def test_an_expert_twice_for_a_token(paro):
    M, E, k, N, d, G = 20, 3, 2, 64, 256, 64
    c = Case(paro, 6, M, E, k, N, d, G)
    ids = np.repeat(np.arange(M)[:, None] % E, k, 1).astype(np.int32)
    weights = c.rng.uniform(0, 1, (M, k)).astype(np.float32)
    r = paro.paro_experts_sort(dev(ids), E, dev(weights))
    offsets, order, _ = experts.tables(ids, E)
    h, dy = c.half(M * k, d), c.half(M, N)
    log("an expert twice")
    y = paro.paro_w4_experts_combine(r, dev(h), *c.dev, bias=c.bd, group=G)
    within(host(y), *experts.combine(offsets, order, k, h, c.w(), c.b, weights, None), "y")
    dh, dw = paro.paro_w4_experts_combine_backward(r, dev(h), *c.dev, dev(dy), bias=c.bd, group=G)
    ref = experts.combine_backward(offsets, order, k, h, c.w(), c.b, weights, dy)
    within(host(dh), ref[0], ref[1], "dh")
    within(host(dw), ref[2], ref[3], "dweights")


def test_every_call_repeats_itself(paro):
    M, E, k, N, d, G = 300, 12, 3, 272, 640, 128
    c = Case(paro, 8, M, E, k, 2 * N, d, G, padded=0.1)
    x, dh = dev(c.half(M, d)), dev(c.half(M * k, N))
    first = None
    for _ in range(3):
        h = paro.paro_w4_experts_gated(c.r, x, *c.dev, bias=c.bd, group=G)[:c.n]
        dx, dz = paro.paro_w4_experts_gated_backward(c.r, x, *c.dev, dh, bias=c.bd, group=G)
        now = (h, dx, dz[:c.n])
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


class Layer:
    """A layer of experts: router, gated block, combining product; forward and backward in the library's calls."""

    def __init__(self, paro, seed, M, E, k, d, H, group=128):
        rng = np.random.default_rng(seed)
        self.paro, self.M, self.E, self.k, self.d, self.H, self.G = paro, M, E, k, d, H, group
        half = lambda *s: dev((rng.standard_normal(s) * 0.05).astype(np.float16))  # noqa: E731
        self.up = [t.view(E, 2 * H, -1) for t in paro.paro_quantize_weights(None, half(E * 2 * H, d), group)]
        self.down = [t.view(E, d, -1) for t in paro.paro_quantize_weights(None, half(E * d, H), group)]
        self.rng = rng

    def forward(self, x, logits):
        r = self.paro.paro_experts_route(logits, self.k)
        h = self.paro.paro_w4_experts_gated(r, x, *self.up, group=self.G)
        return r, h, self.paro.paro_w4_experts_combine(r, h, *self.down, residual=x, group=self.G)

    def backward(self, x, logits, r, h, dy):
        dh, dw = self.paro.paro_w4_experts_combine_backward(r, h, *self.down, dy, group=self.G)
        dx, dz = self.paro.paro_w4_experts_gated_backward(r, x, *self.up, dh, group=self.G)
        return dx, self.paro.paro_experts_route_backward(logits, r.ids, r.weights, dw)

    def inputs(self, n):
        return [(dev(self.rng.standard_normal((self.M, self.d)).astype(np.float16)),
                 dev(self.rng.standard_normal((self.M, self.E)).astype(np.float32)),
                 dev(self.rng.standard_normal((self.M, self.d)).astype(np.float16))) for _ in range(n)]


@pytest.mark.parametrize("M,E,k", [(1, 8, 2), (40, 6, 2), (300, 16, 4)])
def test_layer_gradients_against_differences(paro, M, E, k):
    """A whole layer: the derivative of its fp64 form along random directions."""
    d, H, G = 256, 128, 128
    layer = Layer(paro, M, M, E, k, d, H)
    x, logits, dy = layer.inputs(1)[0]
    log(f"layer M={M} E={E} k={k}")
    r, h, y = layer.forward(x, logits)
    dx, dl = layer.backward(x, logits, r, h, dy)
    up = [block.weights(*(host(t)[e] for t in layer.up), G) for e in range(E)]
    down = [block.weights(*(host(t)[e] for t in layer.down), G) for e in range(E)]
    ids = host(r.ids)
    offsets, order, _ = experts.tables(ids, E)
    xh, lh, g = host(x).astype(np.float64), host(logits).astype(np.float64), host(dy).astype(np.float64)

    def loss(xx, ll):  # the choice of the experts held
        e = np.exp(np.take_along_axis(ll, ids, 1))
        hh, _ = experts.gated(offsets, order, k, xx, up, None, "silu")
        return (experts.combine(offsets, order, k, hh, down, None, e / e.sum(1, keepdims=True), None)[0] * g).sum()
    within(host(y), experts.combine(offsets, order, k, host(h), down, None, host(r.weights), host(x))[0],
           experts.combine(offsets, order, k, host(h), down, None, host(r.weights), host(x))[1], "y")
    for at, grad in ((0, host(dx)), (1, host(dl))):
        u = layer.rng.standard_normal(grad.shape)
        step = 1e-5
        hi = loss(*((xh + step * u, lh) if at == 0 else (xh, lh + step * u)))
        lo = loss(*((xh - step * u, lh) if at == 0 else (xh, lh - step * u)))
        num, own = (hi - lo) / (2 * step), (grad.astype(np.float64) * u).sum()
        # every gradient has the roundings of dh, dz, h (fp16) and its own, 2^-11 each, at random
        size = np.linalg.norm(grad.astype(np.float64) * u)
        assert abs(num - own) < 8 * 2.0 ** -11 * size * 4 + 1e-6, (num, own, size)


@pytest.mark.parametrize("M,E,k", [(1, 8, 2), (3, 4, 4), (64, 8, 2), (90, 5, 3), (500, 8, 2)])
def test_layer_captured(paro, M, E, k):
    """A captured layer, replayed with other inputs (and so other routings), against the eager calls; eager work of
    the same layer and another graph on other buffers in between."""
    layer = Layer(paro, M + 1, M, E, k, 256, 384)
    data = layer.inputs(4)
    log(f"captured layer M={M}")

    def step(x, logits, dy):
        r, h, y = layer.forward(x, logits)
        return (y, *layer.backward(x, logits, r, h, dy))
    want = [step(*d) for d in data]
    graphs = []
    for _ in range(2):
        static = [t.clone() for t in data[0]]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(*static)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*static)
        graphs.append((g, static, out))
    for i in (1, 2, 3, 0, 2):
        for g, static, out in graphs:
            for s, d in zip(static, data[i]):
                s.copy_(d)
            g.replay()
        eager = step(*data[(i + 1) % 4])
        torch.cuda.synchronize()
        for _, _, out in graphs:
            for a, b in zip(out, want[i]):
                assert torch.equal(a, b)
        for a, b in zip(eager, want[(i + 1) % 4]):
            assert torch.equal(a, b)


def test_two_graphs_share_a_workspace(paro):
    """Two captured calls of different sizes on one workspace, replayed in turn on one stream: it is scratch, nothing
    in it outlives a call."""
    layers = [Layer(paro, 5, 40, 6, 2, 256, 384), Layer(paro, 6, 700, 4, 2, 256, 384)]
    data = [layer.inputs(2) for layer in layers]
    ws = torch.randint(0, 255, (1 << 26,), dtype=torch.uint8, device="cuda")
    log("graphs on one workspace")

    def step(layer, x, logits, dy):
        r = paro.paro_experts_route(logits, 2, workspace=ws)
        h = paro.paro_w4_experts_gated(r, x, *layer.up, workspace=ws)
        y = paro.paro_w4_experts_combine(r, h, *layer.down, residual=x, workspace=ws)
        dh, dw = paro.paro_w4_experts_combine_backward(r, h, *layer.down, dy, workspace=ws)
        dx, _ = paro.paro_w4_experts_gated_backward(r, x, *layer.up, dh, workspace=ws)
        return y, dw, dx
    want = [[step(layer, *d) for d in ds] for layer, ds in zip(layers, data)]
    static = [[t.clone() for t in ds[0]] for ds in data]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for layer, st in zip(layers, static):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(layer, *st))
        graphs.append(g)
    for i in (1, 0, 1, 1, 0):
        for st, ds in zip(static, data):
            for a, b in zip(st, ds[i]):
                a.copy_(b)
        for g in graphs:
            g.replay()
        ws.fill_(255)
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w[i]))


def test_layers_on_two_streams(paro):
    layer = Layer(paro, 3, 200, 8, 2, 256, 384)
    data = layer.inputs(2)
    want = [layer.forward(*d[:2])[2] for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for (x, logits, _), st in zip(data, streams):
            r = paro.paro_experts_route(logits, 2, stream=st)
            h = paro.paro_w4_experts_gated(r, x, *layer.up, stream=st)
            got.append((r, h, paro.paro_w4_experts_combine(r, h, *layer.down, residual=x, stream=st)))
        torch.cuda.synchronize()
        for (_, _, y), ref in zip(got, want):
            assert torch.equal(y, ref)


def test_transformed_experts(paro):
    """Experts whose weights carry a shared transform: paro_rotate first, then the products."""
    import synthetic
    M, E, k, d, N = 50, 4, 2, 256, 96
    x, lay, _ = synthetic.linear_case(seed=2, M=M, d=d, N=E * 2 * N, group=128, K=8)
    rot = paro.Rotation(lay.pairs, lay.theta, lay.alpha, 128)
    wq = [t.view(E, 2 * N, -1) for t in paro.paro_quantize_weights(rot, dev(lay.w), 128)]
    r = paro.paro_experts_route(torch.randn((M, E), device="cuda"), k)
    xr = paro.paro_rotate(rot, dev(x))
    h = paro.paro_w4_experts_gated(r, xr, *wq)
    w = [block.weights(*(host(t)[e] for t in wq), 128) for e in range(E)]
    ref, tol = experts.gated(host(r.offsets), host(r.order), k, host(xr), w, None, "silu")
    within(host(h), ref, tol, "h")


def some_rows(c, at):
    """The chosen rows as a routing of their own, each row one token: offsets, order, tokens."""
    expert = np.searchsorted(c.offsets, at, side="right") - 1
    return np.searchsorted(expert, np.arange(c.E + 1)), np.arange(len(at)), c.order[at] // c.k


@pytest.mark.parametrize("M,E,k,N,d", [(262144, 9, 8, 1040, 128), (262144, 9, 8, 64, 1152), (1, 1, 1, 16, 1 << 20),
                                       (1, 1, 1, 1 << 20, 128)])
def test_largest(paro, M, E, k, N, d):
    """More than 2^31 values in h, dz and the sums by row; the widest rows of each side. Some rows are compared."""
    c = Case(paro, M + d, M, E, k, 2 * N, d, 128)
    R = M * k
    rng = np.random.default_rng(1)
    edge = (1 << 31) // max(N, d)
    at = np.unique(np.clip(np.r_[0, edge - 1:edge + 2, edge // 2 - 1:edge // 2 + 2, c.n - 1, rng.integers(0, c.n, 6)],
                           0, c.n - 1))
    offsets, order, tokens = some_rows(c, at)
    normal = lambda *s: torch.randn(s, device="cuda", dtype=torch.float16)  # noqa: E731
    x = normal(M, d)
    w = c.w()
    log(f"largest gated M={M} E={E} k={k} N={N} d={d}")
    h = paro.paro_w4_experts_gated(c.r, x, *c.dev, bias=c.bd)
    ref, tol = experts.gated(offsets, order, 1, host(x[tokens]), w, c.b, "silu")
    within(host(h[at]), ref, tol, "h")
    log("  backward")
    dh = normal(R, N)
    dx, dz = paro.paro_w4_experts_gated_backward(c.r, x, *c.dev, dh, bias=c.bd)
    ref, tol = experts.gated_backward_dz(offsets, order, 1, host(x[tokens]), w, c.b, "silu", host(dh[at]))
    within(host(dz[at]), ref, tol, "dz")
    some = np.unique(tokens[[0, -1]])
    rows = np.concatenate([c.place[m * k:(m + 1) * k] for m in some])
    o, z = np.unique(rows, return_inverse=True)
    so, _, _ = some_rows(c, o)
    pair = np.argsort(z)  # the pairs of the chosen tokens, in row order
    ref, tol = experts.gated_backward_dx(so, pair, k, len(some), w, host(dz[o]))
    within(host(dx[some]), ref, tol, "dx")
    del dx, dz, dh, h, c, x
    torch.cuda.empty_cache()
    c = Case(paro, M + d + 1, M, E, k, N, d, 128)
    w = c.w()
    log("largest combine")
    hh, dy = normal(R, d), normal(M, N)
    y = paro.paro_w4_experts_combine(c.r, hh, *c.dev, bias=c.bd)
    rows = np.concatenate([c.place[m * k:(m + 1) * k] for m in some])
    o, z = np.unique(rows, return_inverse=True)
    so, _, _ = some_rows(c, o)
    pair = np.argsort(z)
    within(host(y[some]), *experts.combine(so, pair, k, host(hh[o]), w, c.b, c.weights[some], None), "y")
    log("  backward")
    dh, dw = paro.paro_w4_experts_combine_backward(c.r, hh, *c.dev, dy, bias=c.bd)
    ref = experts.combine_backward(so, pair, k, host(hh[o]), w, c.b, c.weights[some], host(dy[some]))
    within(host(dh[o]), ref[0], ref[1], "dh")
    within(host(dw[some]), ref[2], ref[3], "dweights")


def test_python_refusals(paro):
    c = Case(paro, 1, 8, 4, 2, 64, 256, 128)
    x = dev(c.half(8, 256))
    with pytest.raises(ValueError):
        paro.paro_w4_experts_gated(c.r, x[:7], *c.dev)  # another number of tokens than the routing's
    with pytest.raises(ValueError):
        paro.paro_w4_experts_gated(c.r, x, *(t[:3] for t in c.dev))  # fewer experts
    with pytest.raises(TypeError):
        paro.paro_w4_experts_gated(c.r, x.float(), *c.dev)
    with pytest.raises(ValueError):
        paro.paro_w4_experts_gated(c.r, x, *c.dev, act="tanh")
    with pytest.raises(ValueError):
        paro.paro_w4_experts_gated(c.r, x, *c.dev, h=torch.empty((16, 16), dtype=torch.float16, device="cuda"))
    with pytest.raises(paro.ParoError):
        paro.paro_w4_experts_combine(c.r, dev(c.half(16, 256)), *c.dev,
                                     workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        paro.paro_experts_route(torch.zeros((2, 4), dtype=torch.float64, device="cuda"), 2)
    with pytest.raises(paro.ParoError):
        paro.paro_experts_route(torch.zeros((2, 4), device="cuda"), 5)
    with pytest.raises(ValueError):
        paro.paro_experts_route(torch.zeros((4, 2), device="cuda").t(), 2)  # not contiguous
    with pytest.raises(TypeError):
        paro.paro_experts_route(torch.zeros((2, 4)), 2)  # on the host
    with pytest.raises(ValueError):
        paro.Routing(c.r.ids, c.r.weights, c.r.offsets, c.r.order[:-1], c.r.place)
    none = paro.paro_experts_route(torch.zeros((0, 4), device="cuda"), 2)
    assert host(none.offsets).tolist() == [0] * 5
    assert paro.paro_w4_experts_gated(none, x[:0], *c.dev).shape == (0, 32)
