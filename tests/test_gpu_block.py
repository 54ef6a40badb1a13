"""Feed-forward products with an epilogue, their gradients and AdamW on the GPU
against the fp64 oracle, value by value, within the bounds that follow from the
documented arithmetic (oracle/block.py)."""
import gc

import numpy as np
import pytest

import oracle
import synthetic
from oracle import block

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
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} against {ref[bad][0]}, bound {np.broadcast_to(tol, ref.shape)[bad][0]}")


class Case:
    """Random codes, scales, zeros, activations and bias of a product."""

    def __init__(self, seed, M, d, rows, group, bias=True):
        rng = np.random.default_rng(seed)
        self.M, self.d, self.rows, self.group, self.rng = M, d, rows, group, rng
        self.x = rng.standard_normal((M, d)).astype(np.float16)
        self.qw = rng.integers(0, 256, (rows, d // 2), dtype=np.uint8)
        self.s = (rng.uniform(0.5, 1.5, (rows, d // group)) * 0.5 / np.sqrt(d)).astype(np.float16)
        self.z = rng.integers(5, 11, (rows, d // group)).astype(np.uint8)
        self.b = (rng.standard_normal(rows) * 0.3).astype(np.float16) if bias else None
        self.dev = [dev(a) for a in (self.qw, self.s, self.z)]
        self.xd, self.bd = dev(self.x), dev(self.b)

    def half(self, *shape):
        return self.rng.standard_normal(shape).astype(np.float16)

    def w(self):
        return block.weights(self.qw, self.s, self.z, self.group)

    def rows_of(self, n=24):
        """Token rows that are checked: all of few, else the ends and a sample."""
        if self.M <= 2 * n:
            return np.arange(self.M)
        mid = self.rng.choice(np.arange(1, self.M - 1), n, replace=False)
        return np.unique(np.concatenate([[0, 63, min(64, self.M - 1), self.M - 1], mid]))


def guarded(M, N, fill=777.0):
    """[M][N] fp16 output inside a larger buffer whose rest must stay as it is."""
    buf = torch.full(((M + 4) * N,), fill, dtype=torch.float16, device="cuda")
    out = buf[2 * N:(M + 2) * N].view(M, N)

    def check():
        torch.cuda.synchronize()
        assert (buf[:2 * N] == fill).all() and (buf[(M + 2) * N:] == fill).all(), "written outside the output"
    return out, check


# every kernel: one k-slice and many, ragged slices, vector and scalar scale
# loads, 1 to 4 blocks of 16 tokens; smaller tiles of each shape with k split
# inside and across workgroups; whole 256 x 256 tiles; stream-K with ranges
# inside one tile and across tiles
SHAPES = [
    (1, 128, 16, 128), (1, 4096, 1024, 128), (2, 640, 80, 64), (3, 512, 48, 256), (4, 1024, 4096, 128),
    (5, 4096, 208, 128), (16, 2560, 1040, 64), (17, 1024, 272, 128), (32, 768, 512, 256), (33, 1536, 144, 128),
    (64, 2048, 1040, 128), (1, 14336, 64, 128), (1, 4096, 8240, 128), (3, 5120, 8208, 128), (13, 4096, 10256, 64),
    (16, 640, 8304, 128), (2, 8192, 8192, 256),
    (65, 128, 16, 128), (70, 1024, 528, 128), (100, 4096, 256, 128), (333, 2560, 1040, 64), (500, 384, 4112, 64),
    (1000, 1024, 2064, 256), (2100, 512, 4368, 128), (2048, 768, 16400, 128),
]
LARGE = [(4096, 1024, 4112, 128), (2048, 8192, 2048, 128), (2600, 8192, 2064, 128), (1300, 8192, 4096, 64)]


def seed_of(*v):
    return sum(int(a) * p for a, p in zip(v, (1, 31, 1009, 7)))


@pytest.mark.parametrize("M,d,N,G", SHAPES + LARGE)
def test_linear_act(paro, M, d, N, G):
    seed = seed_of(M, d, N, G)
    c = Case(seed, M, d, N, G)
    w, at = c.w(), c.rows_of()
    res = c.half(M, N)
    ws = paro.new_workspace(None, M, N, d)
    for i, name in enumerate(block.ACTIVATIONS):
        bias, r = (c.b, res) if i % 2 == 0 else ((None, res) if i == 1 else (c.b, None))
        log(f"linear_act M={M} d={d} N={N} G={G} {name} bias={bias is not None} residual={r is not None}")
        y, check = guarded(M, N)
        paro.paro_w4_linear_act(None, c.xd, *c.dev, bias=dev(bias), residual=dev(r), act=name, y=y, group=G,
                                workspace=ws)
        check()
        rr = None if r is None else r[at]
        within(host(y)[at], block.linear_act(c.x[at], w, bias, rr, name),
               block.linear_tolerance(c.x[at], w, bias, rr, name), name)
    # the residual replaced in place
    y = dev(res)
    paro.paro_w4_linear_act(None, c.xd, *c.dev, bias=c.bd, residual=y, act="silu", y=y, group=G, workspace=ws)
    ref = paro.paro_w4_linear_act(None, c.xd, *c.dev, bias=c.bd, residual=dev(res), act="silu", group=G, workspace=ws)
    assert torch.equal(y, ref)
    # no activation and no residual: paro_w4_linear's values (fewer tokens: sums in another order)
    if M > 1024:
        y = paro.paro_w4_linear_act(None, c.xd, *c.dev, bias=c.bd, group=G, workspace=ws)
        assert torch.equal(y, paro.paro_w4_linear(None, c.xd, *c.dev, bias=c.bd, group=G, workspace=ws))
    assert ws is None or not ws[:16384].any().item(), "arrival counters not left at zero"


@pytest.mark.parametrize("M,d,N,G", [(M, d, max(16, N // 32 * 16), G) for M, d, N, G in SHAPES + LARGE])
def test_gated(paro, M, d, N, G):
    c = Case(seed_of(M, d, N, G) + 1, M, d, 2 * N, G)
    w, at = c.w(), c.rows_of()
    ws = paro.new_gated_workspace(None, M, N, d)
    for i, name in enumerate(block.ACTIVATIONS):
        bias = c.b if i % 2 else None
        log(f"gated M={M} d={d} N={N} G={G} {name} bias={bias is not None}")
        y, check = guarded(M, N)
        paro.paro_w4_gated(None, c.xd, *c.dev, bias=dev(bias), act=name, y=y, group=G, workspace=ws)
        check()
        within(host(y)[at], block.gated(c.x[at], w, bias, name), block.gated_tolerance(c.x[at], w, bias, name), name)
    assert ws is None or not ws[:16384].any().item(), "arrival counters not left at zero"


GRADS = [(1, 128, 16, 128), (2, 640, 80, 64), (16, 1024, 528, 128), (64, 512, 272, 256), (65, 2560, 1040, 64),
         (130, 4096, 256, 128), (333, 768, 2064, 256), (1000, 1024, 4112, 128), (2048, 8192, 2048, 128),
         (2600, 512, 4368, 128),
         (2048, 4096, 4096, 128), (700, 384, 12304, 128), (3, 4096, 8192, 128)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,d,N,G", GRADS)
def test_gradients(paro, M, d, N, G, gated):
    if gated:
        N = max(16, N // 32 * 16)
    rows = 2 * N if gated else N
    c = Case(seed_of(M, d, N, G) + 2, M, d, rows, G)
    w, at = c.w(), c.rows_of()
    dy = c.half(M, N)
    back = paro.paro_w4_gated_backward if gated else paro.paro_w4_linear_act_backward
    ref = block.gated_backward if gated else block.linear_act_backward
    ws = paro.new_gated_backward_workspace(M, N, d) if gated else \
        paro.new_linear_act_backward_workspace(M, N, d, "silu")
    for i, name in enumerate(block.ACTIVATIONS):
        bias = c.b if i % 2 else None
        log(f"backward gated={gated} M={M} d={d} N={N} G={G} {name} bias={bias is not None}")
        own = gated or name != "none"
        dz, check_z = guarded(M, rows)
        dx, check_x = guarded(M, d)
        got_dx, got_dz = back(c.xd, *c.dev, dev(dy), bias=dev(bias), act=name, dz=dz if own else None, dx=dx,
                              group=G, workspace=ws)
        check_z()
        check_x()
        z = dy
        if own:
            _, want = ref(c.x[at], w, bias, name, dy[at])
            z = host(got_dz)
            within(z[at], want, block.grad_tolerance(c.x[at], w, bias, name, dy[at], gated), f"{name} dz")
        else:
            assert got_dz is None
        z = z[at].astype(np.float64)
        within(host(got_dx)[at], z @ w, block.input_grad_tolerance(z, w), f"{name} dx")
    # dz alone
    only, again = back(c.xd, *c.dev, dev(dy), bias=c.bd, act="silu", want_dx=False, group=G, workspace=ws)
    _, full = back(c.xd, *c.dev, dev(dy), bias=c.bd, act="silu", group=G, workspace=ws)
    assert only is None and torch.equal(again, full)
    assert not ws[:16384].any().item(), "arrival counters not left at zero"


# 17 tokens to a few hundred (the gradients from one): every tile shape, ragged in
# tokens and channels, fewer chunks of k than wavefronts and more
TILES = [(17, 128, 16, 64), (20, 2432, 48, 64), (33, 640, 80, 128), (48, 256, 2768, 64), (64, 1024, 2752, 256),
         (30, 1152, 8208, 64), (31, 512, 8240, 256), (100, 2176, 4112, 128), (129, 2048, 4112, 256),
         (250, 2304, 2080, 64), (333, 2560, 1056, 64), (65, 128, 16, 128)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,d,P,G", TILES + [(1, 256, 48, 64), (16, 640, 4112, 128)])
def test_small_tiles(paro, M, d, P, G, gated):
    N = P // 32 * 16 if gated else P
    if N == 0:
        N = 16
    rows = 2 * N if gated else N
    c = Case(seed_of(M, d, P, G) + 9, M, d, rows, G)
    w, at = c.w(), c.rows_of()
    res, dy = c.half(M, N), c.half(M, N)
    for bias, name in [(c.b, "gelu"), (None, "silu")]:
        log(f"small tiles M={M} d={d} N={N} G={G} gated={gated} {name}")
        y, check = guarded(M, N)
        if gated:
            paro.paro_w4_gated(None, c.xd, *c.dev, bias=dev(bias), act=name, y=y, group=G)
            want, tol = block.gated(c.x[at], w, bias, name), block.gated_tolerance(c.x[at], w, bias, name)
        else:
            paro.paro_w4_linear_act(None, c.xd, *c.dev, bias=dev(bias), residual=dev(res), act=name, y=y, group=G)
            want = block.linear_act(c.x[at], w, bias, res[at], name)
            tol = block.linear_tolerance(c.x[at], w, bias, res[at], name)
        check()
        within(host(y)[at], want, tol, name)
        back = paro.paro_w4_gated_backward if gated else paro.paro_w4_linear_act_backward
        ref = block.gated_backward if gated else block.linear_act_backward
        dz, check = guarded(M, rows)
        back(c.xd, *c.dev, dev(dy), bias=dev(bias), act=name, dz=dz, want_dx=False, group=G)
        check()
        within(host(dz)[at], ref(c.x[at], w, bias, name, dy[at])[1],
               block.grad_tolerance(c.x[at], w, bias, name, dy[at], gated), f"{name} dz")


@pytest.mark.parametrize("M", [1, 4, 16, 33, 64, 200])
@pytest.mark.parametrize("group,K", [(128, 8), (64, 3), (256, 8)])
def test_with_transform_equals_transformed_first(paro, M, group, K):
    """A plan r inside the call: the values of paro_rotate's output, the same
    bits beyond 16 tokens (with few, the sums may be taken in another order)."""
    d, N = 1024, 528
    log(f"transform inside M={M} G={group} K={K}")
    x, layer, b = synthetic.linear_case(seed=M + K, M=M, d=d, N=2 * N, group=group, K=K)
    r = paro.Rotation(layer.pairs, layer.theta, layer.alpha, group)
    wq = paro.paro_quantize_weights(r, dev(layer.w), group)
    xd = dev(x)
    xr = paro.paro_rotate(r, xd)
    bd = dev(b)
    res = torch.randn((M, 2 * N), device="cuda").half()
    g = paro.paro_w4_gated(r, xd, *wq, bias=bd, group=group)
    y = paro.paro_w4_linear_act(r, xd, *wq, bias=bd, residual=res, act="gelu_tanh", group=group)
    if M > 16:
        assert torch.equal(g, paro.paro_w4_gated(None, xr, *wq, bias=bd, group=group))
        assert torch.equal(y, paro.paro_w4_linear_act(None, xr, *wq, bias=bd, residual=res, act="gelu_tanh",
                                                      group=group))
    w, xh = block.weights(*(host(t) for t in wq), group), host(xr)
    within(host(g), block.gated(xh, w, b, "silu"), block.gated_tolerance(xh, w, b, "silu"), "gated")
    within(host(y), block.linear_act(xh, w, b, host(res), "gelu_tanh"),
           block.linear_tolerance(xh, w, b, host(res), "gelu_tanh"), "linear")


@pytest.mark.parametrize("M,d,N,group,K", [(1, 4096, 4112, 128, 8), (3, 8192, 1040, 64, 4), (16, 4096, 4112, 128, 8),
                                           (24, 512, 32, 128, 8), (32, 512, 16, 256, 8), (20, 256, 528, 64, 8),
                                           (17, 14336, 640, 128, 8)])
def test_transform_inside_by_size(paro, M, d, N, group, K):
    """A plan r in calls whose transform runs first (2^24 weights, 17 tokens) and
    in those where the workspace leaves no room for X'."""
    log(f"transform by size M={M} d={d} N={N} G={group}")
    x, layer, b = synthetic.linear_case(seed=M + d, M=M, d=d, N=2 * N, group=group, K=K)
    r = paro.Rotation(layer.pairs, layer.theta, layer.alpha, group)
    wq = paro.paro_quantize_weights(r, dev(layer.w), group)
    xd, bd = dev(x), dev(b)
    w, xh = block.weights(*(host(t) for t in wq), group), host(paro.paro_rotate(r, xd))
    wss = paro.new_workspace(r, M, 2 * N, d), paro.new_gated_workspace(r, M, N, d)
    for _ in range(2):
        y = paro.paro_w4_linear_act(r, xd, *wq, bias=bd, act="silu", group=group, workspace=wss[0])
        g = paro.paro_w4_gated(r, xd, *wq, bias=bd, act="gelu", group=group, workspace=wss[1])
        within(host(y), block.linear_act(xh, w, b, None, "silu"), block.linear_tolerance(xh, w, b, None, "silu"), "act")
        within(host(g), block.gated(xh, w, b, "gelu"), block.gated_tolerance(xh, w, b, "gelu"), "gated")
    for ws in wss:
        assert not ws[:16384].any().item(), "arrival counters not left at zero"


# straight from the codes, up to 128 tokens: 1, 2 and 4 blocks of 16 tokens and
# two of 64, one range of weight rows and up to eight, a last chunk of 16, 32 and
# 48 rows, fewer chunks than wavefronts
FEW = [(1, 128, 16, 64), (5, 256, 48, 128), (16, 1024, 4128, 256), (17, 384, 1072, 64), (32, 2560, 8208, 128),
       (33, 4096, 528, 64), (64, 512, 2096, 128), (100, 768, 4112, 256), (128, 8192, 1040, 64), (3, 14336, 1024, 128)]


@pytest.mark.parametrize("M,d,P,G", FEW)
def test_input_gradient_of_few_tokens(paro, M, d, P, G):
    c = Case(seed_of(M, d, P, G) + 11, M, d, P, G)
    w, at = c.w(), c.rows_of()
    dy = c.half(M, P)
    log(f"few tokens M={M} d={d} P={P} G={G}")
    ws = paro.new_linear_act_backward_workspace(M, P, d, "none")
    dx, check = guarded(M, d)
    for _ in range(2):
        paro.paro_w4_linear_act_backward(None, *c.dev, dev(dy), dx=dx, group=G, workspace=ws)
    check()
    z = dy[at].astype(np.float64)
    within(host(dx)[at], z @ w, block.input_grad_tolerance(z, w), "dx")
    # a token that is not finite stays alone, the one behind it included
    bad = dy.copy()
    row = M // 2
    bad[row, ::3], bad[row, 1::3] = np.nan, np.inf
    again = paro.paro_w4_linear_act_backward(None, *c.dev, dev(bad), group=G, workspace=ws)[0]
    keep = np.arange(M) != row
    assert np.array_equal(host(again)[keep], host(dx)[keep]) and not np.isfinite(host(again)[row]).any()


@pytest.mark.parametrize("M", [40, 64])
def test_workspace_of_odd_size(paro, M):
    """A larger workspace of any number of bytes: X' inside it stays aligned."""
    d, N, group = 1024, 256, 128
    x, layer, b = synthetic.linear_case(seed=M, M=M, d=d, N=N, group=group, K=8)
    r = paro.Rotation(layer.pairs, layer.theta, layer.alpha, group)
    wq = paro.paro_quantize_weights(r, dev(layer.w), group)
    xd = dev(x)
    want = paro.paro_w4_linear_act(r, xd, *wq, act="silu", group=group)
    plain = paro.paro_w4_linear(r, xd, *wq, group=group)
    need = paro.paro_w4_linear_workspace_size(r, M, N, d)
    for extra in (1, 3, 14, 255):
        log(f"workspace M={M} extra={extra}")
        ws = torch.zeros(need + extra, dtype=torch.uint8, device="cuda")
        assert torch.equal(paro.paro_w4_linear_act(r, xd, *wq, act="silu", group=group, workspace=ws), want)
        assert torch.equal(paro.paro_w4_linear(r, xd, *wq, group=group, workspace=ws), plain)


def test_not_finite_stays_in_its_row(paro):
    """A token with an infinity or NaN spoils its own outputs only, in every direction."""
    M, d, N = 70, 512, 144   # N is no multiple of 64: the gradient's contraction is padded
    c = Case(17, M, d, 2 * N, 128)
    x, dy = c.x.copy(), c.half(M, N)
    x[3, 5], x[69, 500], dy[10, N - 1], dy[11, 0] = np.inf, np.nan, np.nan, np.inf
    log("not finite")
    y = host(paro.paro_w4_gated(None, dev(x), *c.dev, bias=c.bd))
    bad = ~np.isfinite(y).all(1)
    assert set(np.flatnonzero(bad)) == {3, 69}
    dx, dz = paro.paro_w4_gated_backward(dev(x), *c.dev, dev(dy), bias=c.bd)
    for t in (dx, dz):
        assert set(np.flatnonzero(~np.isfinite(host(t)).all(1))) == {3, 10, 11, 69}
    c = Case(18, M, d, N, 128)
    dx, _ = paro.paro_w4_linear_act_backward(None, *c.dev, dev(dy))
    assert set(np.flatnonzero(~np.isfinite(host(dx)).all(1))) == {10, 11}
    # large pre-activations: the activations saturate without a NaN
    c = Case(19, 8, d, 2 * N, 128)
    x = (c.x.astype(np.float32) * 2000).astype(np.float16)
    for name in block.ACTIVATIONS:
        w = c.w()
        got = host(paro.paro_w4_linear_act(None, dev(x), *c.dev, act=name))
        ref = block.linear_act(x, w, None, None, name)
        tol = block.linear_tolerance(x, w, None, None, name)
        ok = np.abs(ref) < 65000   # above, fp16 overflows to infinity
        within(np.where(ok, got, 0), np.where(ok, ref, 0), np.where(ok, tol, 0), name)
        assert not np.isnan(got).any()


@pytest.mark.parametrize("M", [16, 100, 300, 1100])
def test_streams_and_capture(paro, M):
    """Two streams at once, each with its workspace, and captured calls replayed
    between eager ones, two graphs on one workspace in turn."""
    d, N = 4096, 1024
    c = Case(23 + M, M, d, 2 * N, 128)
    dy = dev(c.half(M, N))
    log(f"streams and capture M={M}")

    def all_calls(wss, stream=None):
        y = paro.paro_w4_gated(None, c.xd, *c.dev, bias=c.bd, workspace=wss[0], stream=stream)
        dx, dz = paro.paro_w4_gated_backward(c.xd, *c.dev, dy, bias=c.bd, workspace=wss[1], stream=stream)
        z = paro.paro_w4_linear_act(None, c.xd, *c.dev, bias=c.bd, act="gelu", workspace=wss[2], stream=stream)
        return y, dx, dz, z

    def spaces():
        return (paro.new_gated_workspace(None, M, N, d), paro.new_gated_backward_workspace(M, N, d),
                paro.new_workspace(None, M, 2 * N, d))

    ref = all_calls(spaces())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [spaces() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = []
        for s, ws in zip(streams, wss):
            with torch.cuda.stream(s):
                outs.append(all_calls(ws))
        torch.cuda.synchronize()
        for out in outs:
            for a, b in zip(out, ref):
                assert torch.equal(a, b)
    ws = spaces()
    gc.collect()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = all_calls(ws)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        outs2 = all_calls(ws)
    for i in range(3):
        for t in outs + outs2:
            t.zero_()
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        for a, a2, b in zip(outs, outs2, ref):
            assert torch.equal(a, b) and torch.equal(a2, b), f"replay {i}"
        for a, b in zip(all_calls(wss[0]), ref):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_workspace_of_one_size_serves_smaller_calls(paro):
    """One workspace for calls of several sizes in a row: the counters stay zero."""
    d = 2048
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    for M, N in [(64, 1024), (1, 64), (300, 512), (16, 1040), (2048, 1024), (4, 16)]:
        log(f"shared workspace M={M} N={N}")
        c = Case(M + N, M, d, 2 * N, 128)
        a = paro.paro_w4_gated(None, c.xd, *c.dev, workspace=ws)
        assert torch.equal(a, paro.paro_w4_gated(None, c.xd, *c.dev))
        dy = dev(c.half(M, N))
        one = paro.paro_w4_gated_backward(c.xd, *c.dev, dy, workspace=ws)
        two = paro.paro_w4_gated_backward(c.xd, *c.dev, dy)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        assert not ws[:16384].any().item()


def test_tensors_are_checked(paro):
    c = Case(29, 4, 256, 64, 128)
    wide = torch.zeros((4, 512), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        paro.paro_w4_linear_act(None, wide[:, ::2], *c.dev)
    with pytest.raises(ValueError, match="shape"):
        paro.paro_w4_linear_act(None, wide, *c.dev)
    with pytest.raises(TypeError):
        paro.paro_w4_linear_act(None, c.xd.float(), *c.dev)
    with pytest.raises(ValueError, match="residual"):
        paro.paro_w4_linear_act(None, c.xd, *c.dev, residual=torch.zeros((4, 32), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="bias"):
        paro.paro_w4_gated(None, c.xd, *c.dev, bias=torch.zeros(32, dtype=torch.float16, device="cuda"))
    with pytest.raises(paro.ParoError):
        paro.paro_w4_linear_act(None, c.xd, *c.dev, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    empty = paro.paro_w4_gated(None, c.xd[:0], *c.dev)
    assert empty.shape == (0, 32)
    dx, dz = paro.paro_w4_gated_backward(c.xd[:0], *c.dev, torch.zeros((0, 32), dtype=torch.float16, device="cuda"))
    assert dx.shape == (0, 256) and dz.shape == (0, 64)


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
LISTS = {"one": [1], "odd": [1, 255, 256, 257, 0, 2047, 2048, 2049, 5000], "many": [3 + 7 * i for i in range(300)],
         "large": [1_500_001, 64]}


def flat_moments(sizes, values):
    """Per-tensor values laid out as the moments are (each tensor padded to 256)."""
    out = []
    for n, a in zip(sizes, values):
        out.append(np.concatenate([a, np.zeros(-n % 256, a.dtype)]))
    return np.concatenate(out) if out else np.zeros(0, np.float32)


def as_f32(t):
    return host(t.float())


@pytest.mark.parametrize("sizes", LISTS)
@pytest.mark.parametrize("ptype,gtype", [("fp32", "fp32"), ("fp32", "fp16"), ("fp16", "fp32"), ("bf16", "bf16"),
                                         ("fp16", "fp16"), ("fp32", "bf16")])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(paro, sizes, ptype, gtype, bits):
    ns = LISTS[sizes]
    log(f"adamw {sizes} {ptype} {gtype} {bits}")
    rng = np.random.default_rng(len(ns) + bits)
    # odd starts inside one buffer: unaligned tensors take the narrow accesses
    odd = sizes in ("odd", "many")

    def tensors(t, scale):
        buf = dev((rng.standard_normal(sum(ns) + 2 * len(ns)) * scale).astype(np.float32)).to(TYPES[t])
        out, at = [], 1 if odd else 0
        for n in ns:
            out.append(buf[at:at + n] if odd else buf[at:at + n].clone())
            at += n + (1 if odd else 0)
        return buf, out

    pbuf, params = tensors(ptype, 1.0)
    _, grads = tensors(gtype, 0.02)
    opt = paro.AdamW(params, grads, state_bits=bits)
    live = np.concatenate([np.arange(n) < n for n in ns] or [[]]).astype(bool)
    m = v = np.zeros(sum(-(-n // 256) * 256 for n in ns), np.float32)
    codes = [np.zeros(m.size, np.uint8)] * 2
    scales = [np.zeros(m.size // 256, np.float32)] * 2
    for step in (1, 2, 3):
        before = pbuf.clone()
        p64 = [as_f32(p).astype(np.float64) for p in params]
        for g in grads:  # another gradient in the same place
            g.mul_(-0.7 if step == 2 else 1.1)
        gs = [as_f32(g) for g in grads]
        flat = flat_moments(ns, gs)
        if bits == 8:
            m = (block.e4m3_values(codes[0]).astype(np.float32).reshape(-1, 256) * scales[0][:, None]).reshape(-1)
            r = (block.e4m3_values(codes[1]).astype(np.float32).reshape(-1, 256) * scales[1][:, None]).reshape(-1)
            v = r * r
        p_all = flat_moments(ns, p64)
        want, _, _ = block.adamw(p_all, flat, m, v, step, **HYPER)
        m, v = block.adamw_moments_f32(flat, m, v, HYPER["betas"])
        opt.step(step, **HYPER)
        torch.cuda.synchronize()
        if bits == 32:
            assert np.array_equal(host(opt.m), m) and np.array_equal(host(opt.v), v)
        else:
            c0, s0 = block.pack_moment(m)
            c1, s1 = block.pack_moment(np.sqrt(v), v > 0)
            got = [host(t.view(torch.uint8)) for t in (opt.m, opt.v)]
            assert np.array_equal(host(opt.m_scale), s0) and np.array_equal(host(opt.v_scale), s1)
            assert np.array_equal(got[1], c1)
            # (a zero's sign may differ)
            assert np.array_equal(np.where(got[0] == 0x80, 0, got[0]), np.where(c0 == 0x80, 0, c0))
            codes, scales = got, [s0, s1]
        half = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[ptype]
        off = 0
        for n, p, old in zip(ns, params, p64):
            ref = want[off:off + n]
            # the parameter: its rounding, and eight fp32 roundings of either
            # term (moments, root, quotient, rate, decay)
            tol = half * np.abs(ref) + 8 * 2.0 ** -24 * (np.abs(old) + 2 * np.abs(ref - old)) + 2.0 ** -25 * (
                ptype == "fp16")
            within(as_f32(p), ref, tol, f"step {step} n={n}")
            off += -(-n // 256) * 256
        if odd:  # what lies between the tensors stays as it was
            keep = torch.ones_like(pbuf, dtype=torch.bool)
            at = 1
            for n in ns:
                keep[at:at + n] = False
                at += n + 1
            assert torch.equal(pbuf[keep], before[keep])


def test_adamw_8bit_edges(paro):
    """Blocks of zeros, tiny and huge values, wide ranges inside a block, and gradients that are not finite."""
    log("adamw 8-bit edges")
    rng = np.random.default_rng(3)
    n = 8 * 256
    g = (rng.standard_normal(n) * np.exp(rng.uniform(-30, 2, n))).astype(np.float32)
    g[:256] = 0.0
    g[256:512] = 1e-35
    g[512:768] *= 1e15
    g[800], g[1100] = np.nan, np.inf
    p = dev(rng.standard_normal(n).astype(np.float32))
    p0 = host(p).copy()
    opt = paro.AdamW([p], [dev(g)], state_bits=8)
    opt.step(1, **HYPER)
    with np.errstate(invalid="ignore"):
        m, v = block.adamw_moments_f32(g, 0 * p0, 0 * p0, HYPER["betas"])
        c0, s0 = block.pack_moment(m)
        c1, s1 = block.pack_moment(np.sqrt(v), v > 0)
    got_m, got_v = (host(t.view(torch.uint8)) for t in (opt.m, opt.v))
    ok = np.ones(n, bool)
    ok[768:1280] = False   # the two blocks with a value that is not finite
    assert np.array_equal((got_m & 0x7F)[ok], (c0 & 0x7F)[ok]) and np.array_equal(got_v[ok], c1[ok])
    assert np.array_equal(host(opt.m_scale), s0, equal_nan=True)
    assert np.array_equal(host(opt.v_scale), s1, equal_nan=True)
    assert not np.isfinite(host(opt.m_scale)[[3, 4]]).any()
    after = host(p)
    assert np.isnan(after[800]) and np.isfinite(np.delete(after, [800, 1100])).all()
    assert np.array_equal(got_v[:256], np.zeros(256)) and np.array_equal(got_m[256:512], np.zeros(256))
    assert (got_v[(v > 0) & ok & np.repeat(s1 > 0, 256)] > 0).all()
    # a second step: the two blocks are NaN as a whole, the others go on
    opt.step(2, **HYPER)
    bad = ~np.isfinite(host(p))
    assert bad[768:1280].all() and not bad[ok].any()


def test_adamw_capture_and_streams(paro):
    log("adamw capture")
    ns = [1000] * 250
    rng = np.random.default_rng(8)
    make = lambda: [dev(rng.standard_normal(n).astype(np.float32)) for n in ns]  # noqa: E731
    a, g = make(), make()
    b = [t.clone() for t in a]
    one, two = paro.AdamW(a, g, state_bits=8), paro.AdamW(b, g, state_bits=8)
    gc.collect()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one.step(5, **HYPER)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        two.step(5, **HYPER, stream=s)
        s.synchronize()
        for x, y in zip(a, b):
            assert torch.equal(x, y), f"replay {i}"
        assert torch.equal(one.m.view(torch.uint8), two.m.view(torch.uint8))
    two.close()
    two.close()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [3, 40, 200])
def test_block_forward_backward_and_step(paro, M):
    """A feed-forward block y = x + down(gated(x)): served, differentiated down to
    both transforms' angles and scales, and stepped."""
    d, N, G, K = 512, 384, 128, 4
    log(f"block M={M}")
    rng = synthetic.rng_for(9000, M)
    layers = []
    for rows, cols in ((2 * N, d), (d, N)):
        w = synthetic.draw_w(rng, rows, cols, 0.05)
        layers.append(synthetic.Layer(w, *synthetic.draw_rotation(rng, cols, G, K), G))
    x = rng.standard_normal((M, d)).astype(np.float16)
    dy = rng.standard_normal((M, d)).astype(np.float16)
    plans = [paro.Rotation(la.pairs, la.theta, la.alpha, G) for la in layers]
    wq = [paro.paro_quantize_weights(r, dev(la.w), G) for r, la in zip(plans, layers)]
    xd, dyd = dev(x), dev(dy)
    h = paro.paro_w4_gated(plans[0], xd, *wq[0])
    y = paro.paro_w4_linear_act(plans[1], h, *wq[1], residual=xd)
    xr = paro.paro_rotate(plans[0], xd)
    dhr, _ = paro.paro_w4_linear_act_backward(None, *wq[1], dyd)
    dh, dth1, dal1 = paro.paro_rotation_backward(plans[1], h, dhr.float())
    dxr, _ = paro.paro_w4_gated_backward(xr, *wq[0], dh.half())
    dx, dth0, dal0 = paro.paro_rotation_backward(plans[0], xd, dxr.float())

    # the same in fp64, without any rounding in between
    w64 = [block.weights(*(host(t) for t in q), G) for q in wq]
    la0, la1 = layers
    xr64 = oracle.rotate_activations(x, la0.pairs, la0.theta, la0.alpha)
    h64 = block.gated(xr64, w64[0], None, "silu")
    hr64 = oracle.rotate_activations(h64, la1.pairs, la1.theta, la1.alpha)
    y64 = x.astype(np.float64) + hr64 @ w64[1].T
    dhr64 = dy.astype(np.float64) @ w64[1]
    dh64, dth1_64, dal1_64 = oracle.rotation_backward(h64, dhr64, la1.pairs, la1.theta, la1.alpha)
    dxr64, _ = block.gated_backward(xr64, w64[0], None, "silu", dh64)
    dx64, dth0_64, dal0_64 = oracle.rotation_backward(x, dxr64, la0.pairs, la0.theta, la0.alpha)
    # at most six roundings to fp16 (2^-11 each) lie on the way to any of
    # these; the gated product's two factors carry each of them at most twice
    for name, got, ref in (("y", y, y64), ("dh", dh, dh64), ("dtheta down", dth1, dth1_64),
                           ("dalpha down", dal1, dal1_64), ("dx", dx, dx64), ("dtheta gated", dth0, dth0_64),
                           ("dalpha gated", dal0, dal0_64)):
        off = np.linalg.norm(host(got).astype(np.float64) - ref) / np.linalg.norm(ref)
        assert off <= 12 * 2.0 ** -11, f"{name}: {off}"

    params = [dev(a) for la in layers for a in (la.theta, la.alpha)]
    grads = [dth0, dal0, dth1, dal1]
    before = [host(p).copy() for p in params]
    opt = paro.AdamW(params, grads, state_bits=8)
    opt.step(1, lr=1e-3, weight_decay=0.0)
    for p, b, g in zip(params, before, grads):
        want, _, _ = block.adamw(b, host(g), 0 * b, 0 * b, 1, 1e-3, (0.9, 0.999), 1e-8, 0.0)
        within(host(p), want, 2.0 ** -24 * np.abs(want) + 8 * 2.0 ** -24 * (np.abs(b) + 2e-3), "stepped")
    # the stepped angles and scales make the next plans
    for la, th, al in zip(layers, params[0::2], params[1::2]):
        r = paro.Rotation(la.pairs, host(th), host(al), G)
        assert r.K == K
        r.close()
