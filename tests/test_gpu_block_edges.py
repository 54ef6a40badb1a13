"""W4 products and AdamW on the GPU where values, sizes and call forms are at an edge."""
import ctypes
import gc
import math
import os
import subprocess
import sys

import numpy as np
import pytest

import synthetic
from oracle import block

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


# ---------------------------------------------------------------------------
# small scales
# ---------------------------------------------------------------------------

class SmallScales:
    """Random codes with scales from 2^-16 to 2^-9: the sixteenth of a scale below 2^-10 is no fp16 number."""

    def __init__(self, rows, d, group):
        rng = np.random.default_rng(rows + d + group)
        self.qw = rng.integers(0, 256, (rows, d // 2), dtype=np.uint8)
        self.s = np.exp2(rng.uniform(-16, -9, (rows, d // group))).astype(np.float16)
        self.z = rng.integers(0, 16, (rows, d // group)).astype(np.uint8)
        self.w = block.weights(self.qw, self.s, self.z, group)
        self.dev = [dev(a) for a in (self.qw, self.s, self.z)]


def one_hot(M, n):
    """[M][n] with 1024 in one column of each row (neighbouring columns: every place of a word of
    codes), and the columns. A product with it is one weight times 2^10, which fp16 holds exactly."""
    cols = (np.arange(M) * 37 + np.arange(M) // 5) % n
    x = np.zeros((M, n), np.float16)
    x[np.arange(M), cols] = 1024.0
    return x, cols


# few tokens (a workgroup per block, and one per CU going from block to block),
# tiles of 16 to 64 tokens, smaller tiles of the large-batch kernels, 256 x 256 tiles
@pytest.mark.parametrize("M,d,N,G", [(1, 512, 64, 128), (4, 1024, 4128, 128), (16, 640, 80, 64), (13, 512, 4112, 256),
                                     (30, 640, 48, 128), (40, 512, 96, 256), (333, 2560, 1040, 64),
                                     (500, 384, 4112, 64), (2048, 768, 16400, 128)])
def test_products_of_small_scales(paro, M, d, N, G):
    log(f"small scales M={M} d={d} N={N} G={G}")
    x, cols = one_hot(M, d)
    xd = dev(x)
    c = SmallScales(N, d, G)
    want = 1024.0 * c.w[:, cols].T
    assert np.array_equal(host(paro.paro_w4_linear(None, xd, *c.dev, group=G)), want), "linear"
    assert np.array_equal(host(paro.paro_w4_linear_act(None, xd, *c.dev, group=G)), want), "linear_act"
    c = SmallScales(2 * N, d, G)
    z = 1024.0 * c.w[:, cols].T
    want = (z[:, :N] * z[:, N:]).astype(np.float16)
    assert np.array_equal(host(paro.paro_w4_gated(None, xd, *c.dev, act="none", group=G)), want), "gated"
    dy = torch.ones((M, N), dtype=torch.float16, device="cuda")
    _, dz = paro.paro_w4_gated_backward(xd, *c.dev, dy, act="none", want_dx=False, group=G)
    assert np.array_equal(host(dz), np.concatenate([z[:, N:], z[:, :N]], 1)), "gated backward"


# straight from the codes in 1, 2 and 4 blocks of 16 tokens, and through the transposed weights
@pytest.mark.parametrize("M,d,P,G", [(1, 512, 48, 64), (16, 256, 1040, 128), (30, 512, 272, 256), (100, 384, 4112, 64),
                                     (300, 512, 1040, 128)])
def test_input_gradient_of_small_scales(paro, M, d, P, G):
    log(f"input gradient of small scales M={M} d={d} P={P} G={G}")
    dy, rows = one_hot(M, P)
    c = SmallScales(P, d, G)
    dx, _ = paro.paro_w4_linear_act_backward(None, *c.dev, dev(dy), group=G)
    assert np.array_equal(host(dx), 1024.0 * c.w[rows])


# ---------------------------------------------------------------------------
# dz where it is dy
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,N", [(1, 16), (3, 80), (130, 1040), (2100, 4112)])
@pytest.mark.parametrize("want_dx", [False, True])
def test_dz_without_activation(paro, M, N, want_dx):
    """Without an activation dZ is dY: a dz that is given receives it, bit for bit, and nothing beside it."""
    log(f"dz without activation M={M} N={N} dx={want_dx}")
    d = 256
    c = SmallScales(N, d, 128)
    dy = torch.from_numpy(np.random.default_rng(M).integers(0, 1 << 16, (M, N), dtype=np.uint16).view(np.int16)).cuda()
    buf = torch.full(((M + 2) * N,), 777, dtype=torch.int16, device="cuda")
    dz = buf[N:(M + 1) * N].view(M, N)
    dx, got = paro.paro_w4_linear_act_backward(None, *c.dev, dy.view(torch.float16), dz=dz.view(torch.float16),
                                               want_dx=want_dx)
    assert (dx is None) == (not want_dx)
    assert torch.equal(got.view(torch.int16), dy) and torch.equal(dz, dy)
    assert (buf[:N] == 777).all() and (buf[(M + 1) * N:] == 777).all()
    # dy itself, and no place at all
    assert paro.paro_w4_linear_act_backward(None, *c.dev, dy.view(torch.float16), dz=dy.view(torch.float16))[1] is not None
    assert torch.equal(dz, dy)
    assert paro.paro_w4_linear_act_backward(None, *c.dev, dy.view(torch.float16))[1] is None


# ---------------------------------------------------------------------------
# infinite pre-activations
# ---------------------------------------------------------------------------

# every kernel with an epilogue: few tokens (both forms), small tiles, smaller
# tiles, 256 x 256 tiles; with a plan (K >= 0) the kernel that transforms as well
@pytest.mark.parametrize("M,d,N,K", [(1, 512, 64, -1), (4, 1024, 4128, -1), (40, 512, 96, -1), (500, 384, 4112, -1),
                                     (2048, 768, 16400, -1), (4, 512, 64, 8)])
def test_infinite_preactivations(paro, M, d, N, K):
    """Z = bias: +inf stays +inf under every activation, and times the other factor of a gated product."""
    log(f"infinite pre-activations M={M} d={d} N={N} K={K}")
    r = None
    if K >= 0:
        _, layer, _ = synthetic.linear_case(seed=K, M=M, d=d, N=N, group=128, K=K)
        r = paro.Rotation(layer.pairs, layer.theta, layer.alpha, 128)
    x = torch.zeros((M, d), dtype=torch.float16, device="cuda")
    c = SmallScales(2 * N, d, 128)
    one = [t[:N].contiguous() for t in c.dev]
    bias = np.zeros(2 * N, np.float16)
    bias[0:N:7], bias[3:N:7] = np.inf, 60000.0            # gate
    bias[N:], bias[N + 1::2] = 2.0, -0.5                   # up
    up, down = np.isposinf(bias[:N]), bias[:N] > 50000
    want_gated = np.where(up, np.where(bias[N:] > 0, np.inf, -np.inf), 0)
    dy = torch.ones((M, N), dtype=torch.float16, device="cuda")
    for act in block.ACTIVATIONS:
        y = host(paro.paro_w4_linear_act(r, x, *one, bias=dev(bias[:N]), act=act))
        assert np.isposinf(y[:, up]).all(), act
        assert (y[:, down & ~up] == np.float16(60000.0)).all() and (y[:, ~down] == 0).all(), act
        g = host(paro.paro_w4_gated(r, x, *c.dev, bias=dev(bias), act=act))
        assert np.array_equal(g[:, up], np.broadcast_to(want_gated[up], (M, up.sum()))), act
        if r is None:  # dzu = dy act(zg)
            _, dz = paro.paro_w4_gated_backward(x, *c.dev, dy, bias=dev(bias), act=act, want_dx=False)
            dzu = host(dz)[:, N:]
            assert np.isposinf(dzu[:, up]).all() and (dzu[:, ~down] == 0).all(), act


# ---------------------------------------------------------------------------
# calls on another stream than the current one
# ---------------------------------------------------------------------------

def spoil(nbytes):
    """Memory of this size on the current stream, full of ones, and freed again."""
    torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("M", [4, 100, 300, 1100])
def test_calls_on_another_stream(paro, M):
    """stream= without a workspace or outputs, while the current stream is busy and hands out memory."""
    d, N = 4096, 1024
    log(f"another stream M={M}")
    x, layer, b = synthetic.linear_case(seed=M, M=M, d=d, N=2 * N, group=128, K=8)
    r = paro.Rotation(layer.pairs, layer.theta, layer.alpha, 128)
    wq = paro.paro_quantize_weights(r, dev(layer.w), 128)
    xd, bd = dev(x), dev(b)
    dy, dy2 = (torch.randn((M, n), device="cuda").half() for n in (N, 2 * N))
    gy = torch.randn((M, d), device="cuda")
    wd = dev(layer.w)

    def calls(**k):
        yield "rotate", lambda: [paro.paro_rotate(r, xd, **k)]
        yield "quantize", lambda: paro.paro_quantize_weights(r, wd, 128, **k)
        yield "linear", lambda: [paro.paro_w4_linear(r, xd, *wq, bias=bd, **k)]
        yield "linear_act", lambda: [paro.paro_w4_linear_act(r, xd, *wq, bias=bd, act="gelu", **k)]
        yield "gated", lambda: [paro.paro_w4_gated(r, xd, *wq, bias=bd, **k)]
        yield "linear_act without a plan", lambda: [paro.paro_w4_linear_act(None, xd, *wq, act="silu", **k)]
        yield "linear_act_backward", lambda: paro.paro_w4_linear_act_backward(xd, *wq, dy2, bias=bd, act="silu", **k)
        yield "gated_backward", lambda: paro.paro_w4_gated_backward(xd, *wq, dy, bias=bd, **k)
        yield "rotation_backward", lambda: paro.paro_rotation_backward(r, xd, gy, **k)
        yield "layer_loss", lambda: paro.paro_layer_loss(r, xd, wd, *wq, **k)

    want = {}
    for name, call in calls():
        want[name] = [t.clone() for t in call()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for name, call in calls(stream=s):
        log(f"  {name}")
        for n in (1 << 16, 1 << 22, 1 << 26):
            spoil(n)
        for _ in range(20):   # (some work that is still running when the call is made)
            gy @ gy.T
        out = call()
        for n in (1 << 16, 1 << 22, 1 << 26):
            spoil(n)          # not into what the call still uses
        s.synchronize()
        for a, w in zip(out, want[name]):
            assert torch.equal(a, w), name
        del out, a
        spoil(1 << 22)
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_made_and_stepped_on_two_streams(paro, bits):
    """A plan made while the current stream is busy, stepped on another one at once, and dropped."""
    log(f"adamw on two streams {bits}")
    n = [100_000] * 3
    rng = np.random.default_rng(bits)
    p0 = [dev(rng.standard_normal(k).astype(np.float32)) for k in n]
    g = [dev(rng.standard_normal(k).astype(np.float32)) for k in n]
    want = [t.clone() for t in p0]
    paro.AdamW(want, g, state_bits=bits).step(1)
    a = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        p = [t.clone() for t in p0]
        torch.cuda.synchronize()
        for k in (1 << 18, 1 << 20, 1 << 21):
            spoil(k)
        for _ in range(10):
            a @ a
        opt = paro.AdamW(p, g, state_bits=bits)
        opt.step(1, stream=s)
        del opt
        for k in (1 << 18, 1 << 20, 1 << 21):
            spoil(k)
        s.synchronize()
        for x, w in zip(p, want):
            assert torch.equal(x, w)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# a plan of another device
# ---------------------------------------------------------------------------

class Plan(ctypes.Structure):
    """The start of a plan as the library keeps it."""
    _fields_ = [("d", ctypes.c_int64), ("group", ctypes.c_int32), ("K", ctypes.c_int32), ("device", ctypes.c_int32),
                ("rest", ctypes.c_int64 * 64)]


def test_plan_of_another_device(paro):
    """Refused with its own error by every product, before anything is enqueued."""
    log("plan of another device")
    d, N = 512, 64
    c = SmallScales(2 * N, d, 128)
    one = [t[:N].contiguous() for t in c.dev]
    y = torch.empty((100, N), dtype=torch.float16, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    plan = Plan(d, 128, 8, torch.cuda.current_device() + 1)

    class Other:
        handle = ctypes.cast(ctypes.pointer(plan), ctypes.c_void_p)

    for M in (4, 100):
        x = torch.zeros((M, d), dtype=torch.float16, device="cuda")
        for call in (lambda: paro.paro_w4_linear(Other, x, *one, y=y[:M], workspace=ws),
                     lambda: paro.paro_w4_linear_noalloc(Other, x, *one, y[:M]),
                     lambda: paro.paro_w4_linear_act(Other, x, *one, y=y[:M], workspace=ws),
                     lambda: paro.paro_w4_gated(Other, x, *c.dev, y=y[:M], workspace=ws)):
            with pytest.raises(paro.ParoError, match="another device") as e:
                call()
            assert e.value.status == -4
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# one plan of steps over the gradients that the library makes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("captured", [False, True])
def test_learning_with_one_plan(paro, captured):
    """Angles and scales of two layers, three steps of one AdamW plan: the gradients of each step are written where
    the plan reads them, eager and replayed."""
    log(f"learning with one plan captured={captured}")
    M, G, K = 96, 128, 4
    layers = []
    for d, N in ((512, 256), (384, 64)):
        x, layer, _ = synthetic.linear_case(seed=d, M=M, d=d, N=N, group=G, K=K)
        r = paro.Rotation(layer.pairs, layer.theta, layer.alpha, G)
        w = dev(layer.w)
        layers.append((r, dev(x), w, paro.paro_quantize_weights(r, w, G), layer))
    theta = [dev(la[4].theta.astype(np.float32)) for la in layers]
    alpha = [dev(la[4].alpha.astype(np.float32)) for la in layers]
    want = [t.clone() for t in theta + alpha]
    dth, dal = [torch.full_like(t, 7) for t in theta], [torch.full_like(t, 7) for t in alpha]
    loss = torch.zeros(1, device="cuda")
    hyper = dict(lr=1e-2, weight_decay=0.0)
    spaces = [torch.zeros(1 << 25, dtype=torch.uint8, device="cuda") for _ in layers]
    gys = [[torch.randn((M, la[4].theta.shape[1] * 2), device="cuda") for la in layers] for _ in range(3)]
    gy = [t.clone() for t in gys[0]]

    def gradients():
        paro.paro_layer_loss(*layers[0][:3], *layers[0][3], loss=loss, dtheta=dth[0], dalpha=dal[0],
                             workspace=spaces[0])
        for a, (r, x, _, _, _), b, c, s in zip(gy[1:], layers[1:], dth[1:], dal[1:], spaces[1:]):
            paro.paro_rotation_backward(r, x, a, dtheta=b, dalpha=c, want_gx=False, workspace=s)

    opt = paro.AdamW(theta + alpha, dth + dal)
    ref = paro.AdamW(want, [torch.zeros_like(t) for t in want])
    graph = None
    if captured:
        gc.collect()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gradients()
    for step in (1, 2, 3):
        for a, b in zip(gy, gys[step - 1]):
            a.copy_(b)
        if graph is not None:
            graph.replay()
        else:
            gradients()
        opt.step(step, **hyper)
        # the same with the gradients made anew and copied
        l0, t0, a0 = paro.paro_layer_loss(*layers[0][:3], *layers[0][3])
        _, t1, a1 = paro.paro_rotation_backward(layers[1][0], layers[1][1], gys[step - 1][1], want_gx=False)
        for to, g in zip(ref.grads, (t0, t1, a0, a1)):
            to.copy_(g)
        ref.step(step, **hyper)
        torch.cuda.synchronize()
        assert torch.equal(loss, l0)
        for got, w in zip(theta + alpha, want):
            assert torch.equal(got, w), step


# ---------------------------------------------------------------------------
# a device that was never set up
# ---------------------------------------------------------------------------

CHILD = r"""
import sys
import torch
sys.path.insert(0, ROOT)
import rotated_w4_linear_amd as paro

gen = torch.Generator(device="cuda").manual_seed(11)
# products over ranges of k in one tile and across tiles; gradients in two and four pieces of 64, 128 and 256 tokens
SHAPES = [(300, 2560, 1040, 64), (1300, 8192, 4096, 64), (2048, 8192, 2048, 128), (192, 4096, 4096, 128),
          (256, 4096, 4096, 128), (1024, 4096, 14336, 128), (2048, 4096, 14336, 128)]
cases = []
for M, d, N, G in SHAPES:
    half = lambda *s: torch.randn(s, generator=gen, device="cuda").half()
    w = [torch.randint(0, 256, (2 * N, d // 2), generator=gen, device="cuda").to(torch.uint8),
         (torch.rand((2 * N, d // G), generator=gen, device="cuda") * 0.01 + 0.002).half(),
         torch.randint(0, 16, (2 * N, d // G), generator=gen, device="cuda").to(torch.uint8)]
    cases.append((M, d, N, G, half(M, d), w, [t[:N].contiguous() for t in w], half(M, N), half(2 * N)))


def results():
    for M, d, N, G, x, w, one, dy, bias in cases:
        print(f"child: M={M} d={d} N={N}", flush=True)
        spaces = (paro.new_workspace(None, M, N, d), paro.new_gated_workspace(None, M, N, d),
                  paro.new_linear_act_backward_workspace(M, N, d, "gelu"), paro.new_gated_backward_workspace(M, N, d))
        y = paro.paro_w4_linear_act(None, x, *one, bias=bias[:N], residual=dy, act="silu", group=G,
                                    workspace=spaces[0])
        g = paro.paro_w4_gated(None, x, *w, bias=bias, group=G, workspace=spaces[1])
        a = paro.paro_w4_linear_act_backward(x, *one, dy, bias=bias[:N], act="gelu", group=G, workspace=spaces[2])
        b = paro.paro_w4_gated_backward(x, *w, dy, bias=bias, group=G, workspace=spaces[3])
        torch.cuda.synchronize()
        for s in spaces:
            assert s is None or not s[:16384].any().item(), "arrival counters not left at zero"
        yield y, g, *a, *b


before = list(results())
paro.paro_device_init()
for i, after in enumerate(results()):
    for p, q in zip(before[i], after):
        assert torch.equal(p, q), SHAPES[i]
print("child: ok", flush=True)
"""


def test_device_that_was_never_set_up():
    """Without paro_device_init the pieces of a split product meet through memory: the same bits as in one XCD's L2."""
    res = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT), 1)], capture_output=True, text=True,
                         timeout=100, cwd=ROOT)
    print(res.stdout, flush=True)
    assert res.returncode == 0, f"child failed ({res.returncode}):\n{res.stdout}\n{res.stderr[-4000:]}"


# ---------------------------------------------------------------------------
# activations value by value
# ---------------------------------------------------------------------------

def act_exactly(name, z):
    """(act, act', a bound of the fp32 evaluation's error of each) in fp64.

    U = 2^-24. The value is z times a factor built from products of positive terms: its relative error is that of
    exp2's argument (2 roundings and a rounded constant: 3 U of the argument, so of 1.44 |u| or 0.72 z^2, times ln 2),
    and at most 64 U for the two ulps of exp2 and rcp each, the polynomial (fit 8 U; eight fused steps over
    coefficients whose magnitudes sum to 1.8 times its value) and the products. The slope is a sum of two such terms,
    the second of which holds 1 - s, off by 2 U of 1.
    """
    U = 2.0 ** -24
    if name == "gelu":
        phi = np.array([0.5 * math.erfc(-v / math.sqrt(2)) for v in z])
        second = z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        rel = (64 + 3 * z * z) * U
        return z * phi, phi + second, rel * np.abs(z * phi), rel * (phi + np.abs(second))
    if name == "relu":
        return np.maximum(z, 0), (z > 0) * 1.0, 0 * z, 0 * z
    a, b = (1.0, 0.0) if name == "silu" else (2 * math.sqrt(2 / math.pi), 2 * math.sqrt(2 / math.pi) * 0.044715)
    u = z * (a + b * z * z)
    s, rest, du = 1 / (1 + np.exp(-u)), 1 / (1 + np.exp(u)), a + 3 * b * z * z
    second = z * s * rest * du
    rel = (64 + 8 * np.abs(u)) * U   # (u itself: 4 roundings and two constants)
    return z * s, s + second, rel * np.abs(z * s), rel * (s + np.abs(second)) + 2 * U * np.abs(z * s * du)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_activations_value_by_value(paro, M, name):
    """Every fp16 number in [-6.5, 6.5] as a pre-activation (the bias; x = 0, so there is no sum to be off): value and
    slope to fp16's own rounding, far out in the tails too."""
    log(f"activation {name} M={M}")
    z = np.arange(1 << 16, dtype=np.uint16).view(np.float16)
    z = z[np.isfinite(z) & (np.abs(z.astype(np.float64)) <= 6.5)]
    N = len(z) // 16 * 16
    z = np.sort(z)[:N]
    d = 128
    w = [dev(a) for a in (np.zeros((N, d // 2), np.uint8), np.ones((N, 1), np.float16), np.zeros((N, 1), np.uint8))]
    x = torch.zeros((M, d), dtype=torch.float16, device="cuda")
    v, dv, ev, edv = act_exactly(name, z.astype(np.float64))
    y = host(paro.paro_w4_linear_act(None, x, *w, bias=dev(z), act=name))
    dy = torch.ones((M, N), dtype=torch.float16, device="cuda")
    _, dz = paro.paro_w4_linear_act_backward(x, *w, dy, bias=dev(z), act=name, want_dx=False)
    for got, ref, err, what in ((y, v, ev, "value"), (host(dz), dv, edv, "slope")):
        tol = 2.0 ** -11 * (np.abs(ref) + err) + 2.0 ** -25 + err
        off = np.abs(got.astype(np.float64) - ref) - tol
        assert (off <= 0).all(), f"{what} at z = {z[np.argmax(off.max(0))]}: {off.max()} beyond the bound"


# ---------------------------------------------------------------------------
# the smallest workspace, plans under capture, the largest sizes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,d,N,G", [(65, 1024, 272, 128), (300, 2560, 1040, 64), (2048, 8192, 2048, 128),
                                     (1300, 8192, 4096, 64)])
def test_products_without_room_for_partial_tiles(paro, M, d, N, G):
    """Beyond 64 tokens without a plan no workspace is needed: k is then not split across workgroups."""
    log(f"no workspace M={M} d={d} N={N}")
    c = SmallScales(2 * N, d, G)
    one = [t[:N].contiguous() for t in c.dev]
    x, cols = one_hot(M, d)
    xd = dev(x)
    z = 1024.0 * c.w[:, cols].T
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    assert np.array_equal(host(paro.paro_w4_linear_act(None, xd, *one, act="relu", group=G, workspace=ws)),
                          np.maximum(z[:, :N], 0))
    assert np.array_equal(host(paro.paro_w4_gated(None, xd, *c.dev, act="none", group=G, workspace=ws)),
                          (z[:, :N] * z[:, N:]).astype(np.float16))
    assert (ws == 0xFF).all()


@pytest.mark.parametrize("M,d,N,G", [(1, 4096, 4128, 128), (16, 2048, 48, 64), (40, 2560, 1040, 64),
                                     (64, 512, 4112, 256)])
def test_products_of_few_tokens_on_the_counters_alone(paro, M, d, N, G):
    """Up to 64 tokens without a plan nothing of a workspace is used, and its first 16 KiB do."""
    log(f"16 KiB workspace M={M} d={d} N={N}")
    c = SmallScales(2 * N, d, G)
    one = [t[:N].contiguous() for t in c.dev]
    x, cols = one_hot(M, d)
    xd = dev(x)
    z = 1024.0 * c.w[:, cols].T
    buf = torch.zeros(2 * 16384, dtype=torch.uint8, device="cuda")
    buf[16384:] = 0xFF
    ws = buf[:16384]
    for _ in range(2):
        assert np.array_equal(host(paro.paro_w4_linear_act(None, xd, *one, act="relu", group=G, workspace=ws)),
                              np.maximum(z[:, :N], 0))
        assert np.array_equal(host(paro.paro_w4_gated(None, xd, *c.dev, act="none", group=G, workspace=ws)),
                              (z[:, :N] * z[:, N:]).astype(np.float16))
    assert not ws.any() and (buf[16384:] == 0xFF).all()
    with pytest.raises(paro.ParoError):
        paro.paro_w4_gated(None, xd, *c.dev, group=G, workspace=ws[:16128])


@pytest.mark.parametrize("M", [1, 16, 24, 64, 300])
@pytest.mark.parametrize("d,N", [(512, 64), (4096, 2064)])
def test_plans_under_capture(paro, M, d, N):
    """The transform inside the activated and gated products, captured and replayed between eager calls."""
    log(f"plan under capture M={M} d={d} N={N}")
    x, layer, b = synthetic.linear_case(seed=M + d, M=M, d=d, N=2 * N, group=128, K=8)
    r = paro.Rotation(layer.pairs, layer.theta, layer.alpha, 128)
    wq = paro.paro_quantize_weights(r, dev(layer.w), 128)
    xd, bd = dev(x), dev(b)
    spaces = paro.new_workspace(r, M, 2 * N, d), paro.new_gated_workspace(r, M, N, d)

    def calls():
        return (paro.paro_w4_linear_act(r, xd, *wq, bias=bd, act="gelu", workspace=spaces[0]),
                paro.paro_w4_gated(r, xd, *wq, bias=bd, workspace=spaces[1]))

    want = [t.clone() for t in calls()]
    gc.collect()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for i in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, w in zip(outs, want):
            assert torch.equal(a, w), f"replay {i}"
        for a, w in zip(calls(), want):
            assert torch.equal(a, w)
        torch.cuda.synchronize()


def test_largest_sizes(paro):
    """Offsets beyond 32 bits: N d just below 2^31 in a gated block, more than 2^31 outputs, 2^21 weight rows."""
    gen = torch.Generator(device="cuda").manual_seed(2)

    def weights(rows, d):
        return [torch.randint(0, 256, (rows, d // 2), generator=gen, device="cuda", dtype=torch.uint8),
                torch.randint(1, 64, (rows, d // 128), generator=gen, device="cuda").half() * 2.0 ** -12,
                torch.randint(0, 16, (rows, d // 128), generator=gen, device="cuda", dtype=torch.uint8)]

    def some(w, rows):  # (q - z) s of these rows
        return block.weights(*(host(t[rows].contiguous()) for t in w), 128)

    d, N = 16256, 1 << 17
    w = weights(2 * N, d)
    at = torch.tensor([0, 1, N // 2 + 5, N - 16, N - 1], device="cuda")
    gate, up = some(w, at), some(w, at + N)
    for M in (1, 40, 200, 600):
        log(f"gated {M} x {d} -> {N}")
        x, cols = one_hot(M, d)
        cols[-1], x[-1] = d - 1, 0
        x[-1, d - 1] = 1024.0
        y = paro.paro_w4_gated(None, dev(x), *w, act="none")
        want = (1024.0 * gate[:, cols] * (1024.0 * up[:, cols])).T.astype(np.float16)
        assert np.array_equal(host(y[:, at]), want)
    del w, y

    M, d, N = 70001, 128, 32768
    log(f"linear_act {M} x {d} -> {N}")
    w = weights(N, d)
    x, cols = one_hot(M, d)
    y = torch.full((M, N), 0.5, dtype=torch.float16, device="cuda")
    paro.paro_w4_linear_act(None, dev(x), *w, residual=y, y=y)
    at = torch.tensor([0, 1, N // 2, N - 1], device="cuda")
    rows = np.array([0, 65535, 65536, M - 2, M - 1])
    want = (1024.0 * some(w, at)[:, cols[rows]] + 0.5).T.astype(np.float16)
    assert np.array_equal(host(y[torch.from_numpy(rows).cuda()][:, at]), want)
    del w, y

    P, d = 1 << 21, 128
    w = weights(P, d)
    for M in (3, 130):
        log(f"input gradient {M} x {P} -> {d}")
        dy = torch.zeros((M, P), dtype=torch.float16, device="cuda")
        rows = torch.arange(M, device="cuda") * 15991 + 5
        rows[-1] = P - 1
        dy[torch.arange(M, device="cuda"), rows] = 1024.0
        dx, _ = paro.paro_w4_linear_act_backward(None, *w, dy)
        assert np.array_equal(host(dx), 1024.0 * some(w, rows))


def test_adamw_of_more_than_2_31_values(paro):
    log("adamw of 2^31 + 1003 values")
    n, tail = (1 << 31) + 1003, 1003 + 2048
    p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), 0.25, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    g[-tail:] = torch.randn(tail, generator=gen, device="cuda").bfloat16()
    p[-tail:] = torch.randn(tail, generator=gen, device="cuda").bfloat16()
    end, gend = p[-tail:].clone(), g[-tail:].clone()
    one, two = paro.AdamW([p], [g], state_bits=8), paro.AdamW([end], [gend], state_bits=8)
    for step in (1, 2):
        one.step(step, lr=0.1)
        two.step(step, lr=0.1)
    torch.cuda.synchronize()
    assert torch.equal(p[-tail:], end)
    assert torch.equal(one.m.view(torch.uint8)[-two.m.numel():], two.m.view(torch.uint8))
    assert torch.equal(one.v_scale[-two.v_scale.numel():], two.v_scale)
    assert (p[:-tail] == p[0]).all()
