"""Feed-forward products, their gradients and AdamW on the CPU: the oracle's
gradients against differences, its number formats against torch's, and every
refusal of the entry points (checked on the host before anything is enqueued)."""
import ctypes

import numpy as np
import pytest

from oracle import block


@pytest.fixture(scope="module")
def paro():
    import rotated_w4_linear_amd as p
    p.load_library()
    return p


def small(seed, M=3, d=128, rows=32):
    rng = np.random.default_rng(seed)
    x, w = rng.standard_normal((M, d)), rng.standard_normal((rows, d)) * 0.1
    return rng, x, w, rng.standard_normal(rows) * 0.1


@pytest.mark.parametrize("name", block.ACTIVATIONS)
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_against_differences(name, gated):
    rng, x, w, b = small(3 + gated)
    n = w.shape[0] // 2 if gated else w.shape[0]
    dy = rng.standard_normal((x.shape[0], n))
    fwd = (lambda x_, b_: block.gated(x_, w, b_, name)) if gated else (
        lambda x_, b_: block.linear_act(x_, w, b_, None, name))
    dx, dz = (block.gated_backward if gated else block.linear_act_backward)(x, w, b, name, dy)
    h = 1e-5
    for _ in range(20):
        i, j = rng.integers(x.shape[0]), rng.integers(x.shape[1])
        e = np.zeros_like(x)
        e[i, j] = h
        num = ((fwd(x + e, b) - fwd(x - e, b)) * dy).sum() / (2 * h)
        assert abs(num - dx[i, j]) < 1e-7 * (1 + abs(num))
        k = rng.integers(len(b))
        e = np.zeros_like(b)
        e[k] = h
        num = ((fwd(x, b + e) - fwd(x, b - e)) * dy).sum() / (2 * h)
        assert abs(num - dz[:, k].sum()) < 1e-7 * (1 + abs(num))


def test_slopes_stay_below_the_bounds_the_tolerances_use():
    z = np.linspace(-12, 12, 200001)
    for name in block.ACTIVATIONS:
        s = block.act_grad(name, z)
        assert np.abs(s).max() <= block.SLOPE
        if name != "relu":
            assert np.abs(np.diff(s) / np.diff(z)).max() <= block.BEND


def test_e4m3_rounding_equals_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(5)
    x = (np.exp(rng.uniform(-14, 6.1, 50000)) * rng.choice([-1, 1], 50000)).astype(np.float32)
    x = np.concatenate([x, block.E4M3, (block.E4M3[1:] + block.E4M3[:-1]) / 2, [0.0, -0.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn)
    got = block.e4m3_codes(x)
    assert np.array_equal(got, want.view(torch.uint8).numpy())
    assert np.array_equal(block.e4m3_values(got), want.double().numpy())


D = ctypes.c_void_p(16 * 1024)
ODD = ctypes.c_void_p(16 * 1024 + 8)


def test_linear_act_refusals(paro):
    f = paro.load_library().paro_w4_linear_act

    def call(x=D, q=D, s=D, z=D, b=None, res=None, act=1, y=D, M=4, N=64, d=256, G=128, ws=None, nb=0):
        return f(None, x, q, s, z, b, res, act, y, M, N, d, G, ws, nb, None)

    assert call(act=5) == -4 and call(act=-1) == -4
    assert call(x=None) == -1 and call(y=None) == -1
    assert call(res=ODD) == -5 and call(x=ODD) == -5
    assert call(N=60) == -2 and call(d=200) == -2 and call(M=-1) == -2
    assert call(G=32) == -6 and call(M=1 << 31) == -6
    assert call() == -7                                  # small batches need the counters
    assert call(ws=ODD, nb=1 << 30) == -5                # workspace 256-byte aligned
    assert call(M=0) == 0


def test_gated_refusals(paro):
    lib = paro.load_library()

    def call(x=D, act=1, y=D, M=4, N=64, d=256, G=128, ws=None, nb=0):
        return lib.paro_w4_gated(None, x, D, D, D, None, act, y, M, N, d, G, ws, nb, None)

    assert call(act=9) == -4 and call(x=None) == -1 and call(y=ODD) == -5
    assert call(N=24) == -2 and call(N=0) == -2 and call(N=-16) == -2   # 2 N alone would pass with N = 24
    assert call(N=1 << 20, d=4096) == -6                                 # N d < 2^31
    assert call() == -7 and call(M=0) == 0
    assert lib.paro_w4_gated_workspace_size(None, 4, 64, 1024) == \
        lib.paro_w4_linear_workspace_size(None, 4, 128, 1024)
    assert lib.paro_w4_gated_workspace_size(None, 4, 1 << 40, 1024) == 0


def test_backward_refusals(paro):
    lib = paro.load_library()
    for f, gated in ((lib.paro_w4_linear_act_backward, False), (lib.paro_w4_gated_backward, True)):
        def call(x=D, act=1, dy=D, dz=D, dx=D, M=4, N=64, d=256, G=128, ws=None, nb=0):
            return f(x, D, D, D, None, act, dy, dz, dx, M, N, d, G, ws, nb, None)

        assert call(act=5) == -4
        assert call(x=None) == -1 and call(dy=None) == -1 and call(dz=None) == -1
        assert call(dy=ODD) == -5 and call(dx=ODD) == -5 and call(dz=ODD) == -5
        assert call(N=40) == -2 and call(d=100) == -2
        assert call(N=1 << 23) == -6
        assert call() == -7 and call(ws=ODD, nb=1 << 30) == -5
        assert call(M=0) == 0
        size = (lambda *a: lib.paro_w4_gated_backward_workspace_size(*a)) if gated else (
            lambda *a: lib.paro_w4_linear_act_backward_workspace_size(*a, 1))
        assert size(0, 64, 256) == 0 and size(4, -1, 256) == 0
        assert call(ws=ctypes.c_void_p(1 << 20), nb=size(4, 64, 256) - 1) == -7
    # without activation neither x nor dz nor a product's workspace is needed
    f = lib.paro_w4_linear_act_backward
    assert f(None, D, D, D, None, 0, D, None, D, 4, 64, 256, 128, None, 0, None) == -7
    assert f(None, D, D, D, None, 0, D, None, None, 4, 64, 256, 128, None, 0, None) == 0  # nothing asked for


def adamw_create(paro, n, params, grads, ptype=0, gtype=0, bits=32, m=1 << 24, v=1 << 26, ms=None, vs=None):
    lib = paro.load_library()
    arr = lambda t, a: np.ascontiguousarray(np.asarray(a, t))  # noqa: E731
    n_, p_, g_ = arr(np.int64, n), arr(np.uint64, params), arr(np.uint64, grads)
    h = ctypes.c_void_p()
    vp = lambda a: ctypes.c_void_p(a) if a else None  # noqa: E731
    st = lib.paro_adamw_create(len(n_), paro._ptr(n_), paro._ptr(p_), ptype, paro._ptr(g_), gtype, bits, vp(m), vp(v),
                               vp(ms), vp(vs), ctypes.byref(h))
    return st, h


def test_adamw_refusals(paro):
    lib = paro.load_library()
    P, G = 1 << 16, 1 << 18
    ok = ([300, 0, 5], [P, 0, P + 4096], [G, 0, G + 4096])
    st, h = adamw_create(paro, *ok)
    assert st == 0 and h.value
    for bad in (dict(step=0), dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0), dict(b2=-0.1), dict(eps=0.0),
                dict(eps=float("inf")), dict(wd=-1.0), dict(b1=float("nan"))):
        a = dict(step=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0) | bad
        assert lib.paro_adamw_step(h, a["step"], a["lr"], a["b1"], a["b2"], a["eps"], a["wd"], None) == -4, bad
    # rates that fp32 does not hold: refused, not stepped to infinity
    assert lib.paro_adamw_step(h, 1, 1e300, 0.9, 0.999, 1e-8, 0.0, None) == -4
    assert lib.paro_adamw_step(h, 1, 1e20, 0.9, 0.999, 1e-8, 1e20, None) == -4
    assert lib.paro_adamw_step(None, 1, 1e-3, 0.9, 0.999, 1e-8, 0.0, None) == -1
    lib.paro_adamw_destroy(h)
    lib.paro_adamw_destroy(None)
    assert adamw_create(paro, *ok, ptype=3)[0] == -4 and adamw_create(paro, *ok, gtype=-1)[0] == -4
    assert adamw_create(paro, *ok, bits=16)[0] == -6
    assert adamw_create(paro, *ok, m=0)[0] == -1
    assert adamw_create(paro, *ok, bits=8)[0] == -1                               # scales missing
    assert adamw_create(paro, *ok, m=(1 << 24) + 8)[0] == -5
    assert adamw_create(paro, [-1], [P], [G])[0] == -2
    assert adamw_create(paro, [4], [0], [G])[0] == -1
    assert adamw_create(paro, [4], [P + 2], [G])[0] == -5
    assert adamw_create(paro, [4, 4], [P, P], [G, G + 64])[0] == -4               # the same tensor twice
    assert adamw_create(paro, [400, 4], [P, P + 1596], [G, G + 4096])[0] == -4    # overlapping by one value
    assert adamw_create(paro, [400], [P], [P + 1596])[0] == -4                    # a gradient inside a parameter
    assert adamw_create(paro, [400], [P], [P - 4])[0] == -4
    assert adamw_create(paro, [4], [P], [G], v=(1 << 24) + 512)[0] == -4          # moments overlap
    # gradients may be shared, and empty lists and tensors are no-ops
    st, h = adamw_create(paro, [4, 4], [P, P + 64], [G, G])
    assert st == 0
    lib.paro_adamw_destroy(h)
    st, h = adamw_create(paro, [0], [0], [0], m=0, v=0)
    assert st == 0 and lib.paro_adamw_step(h, 1, 1e-3, 0.9, 0.999, 1e-8, 0.0, None) == 0
    lib.paro_adamw_destroy(h)


def test_adamw_moments(paro):
    assert paro.paro_adamw_moments([]) == 0
    assert paro.paro_adamw_moments([1, 256, 257, 0]) == 256 + 256 + 512
    with pytest.raises(ValueError):
        paro.paro_adamw_moments([-1])


def test_python_refusals(paro):
    import torch
    with pytest.raises(ValueError, match="act"):
        paro._act("swish")
    with pytest.raises(TypeError):
        paro._expect(torch.zeros(4), "x", (4,), torch.float32, 0)   # not a device tensor
    with pytest.raises(ValueError):
        paro.AdamW([], [])
