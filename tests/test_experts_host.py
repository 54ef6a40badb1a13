"""The experts' operators and the distillation loss on the CPU: the oracle's gradients
against differences, and every refusal of the entry points (checked on the host before
anything is enqueued)."""
import ctypes

import numpy as np
import pytest

from oracle import experts
from test_block_edges_host import FakeStream, FakeTensor, fake, faked, paro  # noqa: F401


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

def difference(f, x, at, h):
    a, b = x.copy(), x.copy()
    a[at] += h
    b[at] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("normalize", [False, True])
def test_route_gradient_against_differences(normalize):
    rng = np.random.default_rng(3)
    x, dw = rng.standard_normal((4, 9)), rng.standard_normal((4, 3))
    x[1, 4:] = -np.inf
    x[3] = -np.inf
    ids, w = experts.route(x, 3, normalize)
    grad, _ = experts.route_backward(x, ids, w, dw, normalize)

    def value(a):  # the choice of the experts held
        with np.errstate(invalid="ignore"):
            e = np.exp(a - a.max(1, keepdims=True))
        e = np.nan_to_num(e)
        taken = np.take_along_axis(e, np.maximum(ids, 0), 1) * (ids >= 0)
        total = taken.sum(1) if normalize else e.sum(1)
        return (taken * dw).sum(1) / np.maximum(total, 1e-300)
    for m, j in [(0, 0), (0, 5), (1, 2), (2, 8), (2, 1)]:
        num = difference(lambda a: value(a).sum(), x, (m, j), 1e-6)
        assert abs(num - grad[m, j]) < 1e-8
    assert not grad[3].any()


def stack(rng, E, P, d):
    return [rng.standard_normal((P, d)) * 0.1 for _ in range(E)]


def test_products_gradients_against_differences():
    rng = np.random.default_rng(5)
    M, E, k, d, N = 4, 3, 2, 24, 6
    ids = np.array([[0, 2], [2, -1], [-1, -1], [1, 0]])
    offsets, order, place = experts.tables(ids, E)
    x, dh = rng.standard_normal((M, d)), rng.standard_normal((M * k, N))
    wg, bg = stack(rng, E, 2 * N, d), rng.standard_normal((E, 2 * N)) * 0.1
    dz, _ = experts.gated_backward_dz(offsets, order, k, x, wg, bg, "silu", dh)
    dx, _ = experts.gated_backward_dx(offsets, order, k, M, wg, dz)
    n = offsets[-1]

    def value(a):
        return (experts.gated(offsets, order, k, a, wg, bg, "silu")[0] * dh)[:n].sum()
    for at in [(0, 0), (1, 3), (3, 23)]:
        assert abs(difference(value, x, at, 1e-5) - dx[at]) < 1e-7
    assert not dx[2].any()
    wd, bd = stack(rng, E, N, d), rng.standard_normal((E, N))
    h, weights, dy = rng.standard_normal((M * k, d)), rng.uniform(0, 1, (M, k)), rng.standard_normal((M, N))
    dhid, _, dw, _ = experts.combine_backward(offsets, order, k, h, wd, bd, weights, dy)

    def down(hh, ww):
        return (experts.combine(offsets, order, k, hh, wd, bd, ww, None)[0] * dy).sum()
    for at in [(0, 0), (n - 1, 5)]:
        assert abs(difference(lambda a: down(a, weights), h, at, 1e-5) - dhid[at]) < 1e-7
    for at in [(0, 0), (0, 1), (1, 0), (3, 1)]:
        assert abs(difference(lambda a: down(h, a), weights, at, 1e-5) - dw[at]) < 1e-7
    assert dw[1, 1] == 0 and not dw[2].any()


@pytest.mark.parametrize("rest", [False, True])
def test_distill_gradient_against_differences(rest):
    rng = np.random.default_rng(7)
    M, V, K, T = 3, 13, 4, 2.0
    z, t = rng.standard_normal((M, V)), rng.standard_normal((M, V)) * 2
    index = np.argsort(-t, 1)[:, :K].copy()
    index[0, 1] = index[0, 0]  # the same index twice
    index[1, 2] = -1
    values = np.take_along_axis(t, np.maximum(index, 0), 1)
    if rest:
        values[0, 1] -= 3.0
    lse = np.log(np.exp(t / T).sum(1)) + 0.3 if rest else None
    w = np.array([1.0, 0.5, 2.0])

    def value(a):
        return experts.distill(a, values, index, lse, w, T, 1.0, "fp32")[0].sum()
    dz = experts.distill(z, values, index, lse, w, T, 1.0, "fp32")[2]
    for m in range(M):
        for j in range(V):
            assert abs(difference(value, z, (m, j), 1e-6) - dz[m, j]) < 1e-8


def test_distill_loss_is_zero_between_equals():
    rng = np.random.default_rng(9)
    z = rng.standard_normal((2, 11)) * 3
    index = np.argsort(-z, 1)[:, :4]
    values = np.take_along_axis(z, index, 1)
    lse = np.log(np.exp(z).sum(1))
    loss, _, dz, _ = experts.distill(z, values, index, lse, None, 1.0, 1.0, "fp32")
    assert np.abs(loss).max() < 1e-14 and np.abs(dz).max() < 1e-15


# ---------------------------------------------------------------------------
# refusals: nothing is enqueued, so addresses need not be real ones
# ---------------------------------------------------------------------------

A = 0x10000  # an aligned address
NULL, SHAPE, VALUE, ALIGN, UNSUPPORTED, WORKSPACE = -1, -2, -4, -5, -6, -7


def refused(paro, fn, args, status):
    assert fn(*args) == status, paro.load_library().paro_last_error()
    assert paro.load_library().paro_last_error()


def test_route_refusals(paro):
    lib = paro.load_library()

    def args(logits=A, type=0, M=1000, E=8, k=2, normalize=1, ids=A, weights=A, offsets=A, order=A, place=A, ws=A,
             ws_bytes=1 << 20):
        return logits, type, M, E, k, normalize, ids, weights, offsets, order, place, ws, ws_bytes, None
    fn = lib.paro_experts_route
    for bad, status in [({"logits": None}, NULL), ({"ids": None}, NULL), ({"weights": None}, NULL),
                        ({"offsets": None}, NULL), ({"order": None}, NULL), ({"place": None}, NULL),
                        ({"type": 3}, VALUE), ({"type": -1}, VALUE), ({"M": -1}, SHAPE), ({"E": 0}, SHAPE),
                        ({"k": 0}, SHAPE), ({"k": 9}, SHAPE), ({"E": 1025}, UNSUPPORTED),
                        ({"E": 64, "k": 17}, UNSUPPORTED), ({"M": 1 << 30}, UNSUPPORTED),
                        ({"M": 1 << 23}, UNSUPPORTED),
                        ({"logits": A + 2}, ALIGN), ({"ids": A + 2}, ALIGN), ({"ws": None}, WORKSPACE),
                        ({"ws_bytes": 17}, WORKSPACE), ({"ws": A + 128}, ALIGN)]:
        refused(paro, fn, args(**bad), status)
    assert lib.paro_experts_route_workspace_size(128, 8, 2) == 0
    assert lib.paro_experts_route_workspace_size(129, 8, 2) == 3 * 10 * 2
    for M, E, k in [(-1, 8, 2), (10, 0, 1), (10, 8, 9), (100, 2000, 2), (1 << 30, 8, 2)]:
        assert lib.paro_experts_route_workspace_size(M, E, k) == 0

    sort = lib.paro_experts_sort
    ok = [A, 1000, 8, 2, A, A, A, A, 1 << 20, None]
    for i, v, status in [(0, None, NULL), (4, None, NULL), (5, None, NULL), (6, None, NULL), (1, -1, SHAPE),
                         (2, 0, SHAPE), (3, 17, SHAPE), (7, None, WORKSPACE), (0, A + 2, ALIGN)]:
        refused(paro, sort, ok[:i] + [v] + ok[i + 1:], status)

    back = lib.paro_experts_route_backward
    ok = [A, 0, 100, 8, 2, 0, A, A, A, A, None]
    for i, v, status in [(0, None, NULL), (6, None, NULL), (7, None, NULL), (8, None, NULL), (9, None, NULL),
                         (1, 7, VALUE), (3, 0, SHAPE), (9, A + 2, ALIGN), (8, A + 1, ALIGN)]:
        refused(paro, back, ok[:i] + [v] + ok[i + 1:], status)
    assert back(None, 0, 0, 8, 2, 1, None, None, None, None, None) == 0


def routing(paro, M=100, E=8, k=2, **tables):
    t = {name: A for name in ("ids", "offsets", "order", "place", "weights")}
    t.update(tables)
    return paro._Routing(M, E, k, *(t[n] for n in ("ids", "offsets", "order", "place", "weights")))


SIZES = dict(N=64, d=256, group=128)


def product_args(call, r, x=A, qw=A, sc=A, zr=A, bias=A, act=1, aux=A, out=A, out2=A, N=64, d=256, group=128, ws=A,
                 ws_bytes=1 << 40):
    p = ctypes.byref(r) if r is not None else None
    head = (p, x, qw, sc, zr, bias)
    tail = (N, d, group, ws, ws_bytes, None)
    if call == "gated":
        return head + (act, out) + tail
    if call == "combine":
        return head + (aux, out) + tail
    return head + ((act,) if call == "gated_backward" else ()) + (aux, out, out2) + tail


CALLS = ["gated", "combine", "gated_backward", "combine_backward"]


@pytest.mark.parametrize("call", CALLS)
def test_product_refusals(paro, call):
    fn = getattr(paro.load_library(), f"paro_w4_experts_{call}")
    r = routing(paro)
    refused(paro, fn, product_args(call, None), NULL)
    for bad, status in [({"x": None}, NULL), ({"qw": None}, NULL), ({"sc": None}, NULL), ({"zr": None}, NULL),
                        ({"out": None}, NULL), ({"N": 0}, SHAPE), ({"N": 24}, SHAPE), ({"N": -16}, SHAPE),
                        ({"d": 64}, SHAPE), ({"d": 0}, SHAPE), ({"d": 128, "group": 256}, SHAPE),
                        ({"group": 32}, UNSUPPORTED), ({"N": 1 << 22}, UNSUPPORTED), ({"d": 1 << 22}, UNSUPPORTED),
                        ({"N": 1 << 16, "d": 1 << 15}, UNSUPPORTED), ({"x": A + 8}, ALIGN), ({"qw": A + 8}, ALIGN),
                        ({"sc": A + 2}, ALIGN), ({"zr": A + 4}, ALIGN), ({"bias": A + 8}, ALIGN),
                        ({"out": A + 8}, ALIGN), ({"ws": A + 16}, ALIGN)]:
        refused(paro, fn, product_args(call, r, **bad), status)
    for name in ("ids", "offsets", "order", "place"):
        refused(paro, fn, product_args(call, routing(paro, **{name: None})), NULL)
        refused(paro, fn, product_args(call, routing(paro, **{name: A + 2})), ALIGN)
    for M, E, k, status in [(-1, 8, 2, SHAPE), (10, 0, 1, SHAPE), (10, 4, 5, SHAPE), (10, 2000, 2, UNSUPPORTED),
                            (10, 64, 17, UNSUPPORTED), (1 << 30, 8, 2, UNSUPPORTED), (1 << 23, 8, 2, UNSUPPORTED)]:
        refused(paro, fn, product_args(call, routing(paro, M=M, E=E, k=k)), status)
    # limits that keep every grid below 2^32 lanes
    big = dict(N=1 << 16, d=1 << 13) if call.startswith("gated") else dict(N=1 << 17, d=1 << 13)
    refused(paro, fn, product_args(call, routing(paro, M=100, E=1024), **big), UNSUPPORTED)  # E P = 2^27
    wide = dict(N=128, d=1 << 16) if call.startswith("gated") else dict(N=1 << 12, d=1 << 16)
    refused(paro, fn, product_args(call, routing(paro, M=1 << 14, k=16, E=16), **wide), UNSUPPORTED)  # R d = 2^34
    if call != "gated":
        refused(paro, fn, product_args(call, r, ws=None), WORKSPACE)
        refused(paro, fn, product_args(call, r, ws_bytes=255), WORKSPACE)
    if call.startswith("gated"):
        for act in (-1, 5):
            refused(paro, fn, product_args(call, r, act=act), VALUE)
    else:
        refused(paro, fn, product_args(call, routing(paro, weights=None)), NULL)
        refused(paro, fn, product_args(call, r, aux=A + 8), ALIGN)
    if call.endswith("backward"):
        refused(paro, fn, product_args(call, r, aux=None), NULL)
        refused(paro, fn, product_args(call, r, out2=A + 2), ALIGN)
    if call == "combine_backward":
        refused(paro, fn, product_args(call, r, out2=None), NULL)
    # no tokens: nothing to do, whatever the tensors
    none = routing(paro, M=0, ids=None, offsets=None, order=None, place=None, weights=None)
    assert fn(*product_args(call, none, x=None, qw=None, sc=None, zr=None, bias=None, aux=None, out=None, out2=None,
                            ws=None, ws_bytes=0)) == 0


@pytest.mark.parametrize("call", CALLS)
def test_workspace_sizes_of_refused_sizes(paro, call):
    size = getattr(paro.load_library(), f"paro_w4_experts_{call}_workspace_size")
    for M, E, k, N, d in [(0, 8, 2, 64, 256), (-1, 8, 2, 64, 256), (10, 0, 2, 64, 256), (10, 8, 0, 64, 256),
                          (10, 8, 9, 64, 256), (10, 8, 2, 0, 256), (10, 8, 2, 24, 256), (10, 8, 2, 64, 0),
                          (10, 8, 2, 64, 64), (10, 8, 2, 1 << 40, 256), (10, 8, 2, 64, 1 << 40),
                          (1 << 40, 8, 2, 64, 256), (10, 2000, 2, 64, 256), (1 << 23, 8, 2, 64, 256),
                          (10, 1024, 2, 1 << 17, 1 << 13), (1 << 14, 16, 16, 128, 1 << 16)]:
        assert size(M, E, k, N, d) == 0, (M, E, k, N, d)
    if call != "gated":
        assert size(10, 8, 2, 64, 256) >= 10 * 2 * 4 * (256 if call.endswith("backward") else 64)


def test_distill_refusals(paro):
    fn = paro.load_library().paro_distill_loss

    def args(z=A, zt=0, values=A, vt=0, index=A, lse=A, w=A, M=4, V=100, K=8, T=1.0, scale=1.0, loss=A, dz=A):
        return z, zt, values, vt, index, lse, w, M, V, K, T, scale, loss, dz, None
    inf, nan = float("inf"), float("nan")
    for bad, status in [({"z": None}, NULL), ({"values": None}, NULL), ({"index": None}, NULL), ({"loss": None}, NULL),
                        ({"zt": 3}, VALUE), ({"vt": -1}, VALUE), ({"T": 0.0}, VALUE), ({"T": -1.0}, VALUE),
                        ({"T": inf}, VALUE), ({"T": nan}, VALUE), ({"T": 1e-60}, VALUE), ({"T": 1e-42}, VALUE),
                        ({"scale": inf}, VALUE), ({"scale": 1e40}, VALUE), ({"M": -1}, SHAPE), ({"V": 0}, SHAPE),
                        ({"K": 0}, SHAPE), ({"K": 1025}, UNSUPPORTED), ({"V": (1 << 20) + 1}, UNSUPPORTED),
                        ({"M": 1 << 31}, UNSUPPORTED), ({"M": 1 << 22}, UNSUPPORTED), ({"z": A + 4}, ALIGN), ({"dz": A + 8}, ALIGN),
                        ({"values": A + 2}, ALIGN), ({"index": A + 2}, ALIGN), ({"lse": A + 1}, ALIGN),
                        ({"w": A + 2}, ALIGN), ({"loss": A + 2}, ALIGN)]:
        refused(paro, fn, args(**bad), status)
    assert fn(*args(z=None, values=None, index=None, loss=None, dz=None, M=0)) == 0


# ---------------------------------------------------------------------------
# calls on another stream or device: where their memory is made, what is refused
# ---------------------------------------------------------------------------

def with_routing(call):
    def run(p, **k):
        r = p.Routing(fake(4, 2), fake(4, 2), fake(9), fake(8), fake(8))
        return call(p, r, **k)
    return run


BLOCK = lambda: (fake(8, 64, 128), fake(8, 64, 2), fake(8, 64, 2))  # noqa: E731
STREAM_CALLS = {
    "route": lambda p, **k: p.paro_experts_route(fake(4, 8), 2, **k)._table,
    "sort": lambda p, **k: p.paro_experts_sort(fake(4, 2), 8, fake(4, 2), **k)._table,
    "route_backward": lambda p, **k: p.paro_experts_route_backward(fake(4, 8), fake(4, 2), fake(4, 2), fake(4, 2), **k),
    "gated": with_routing(lambda p, r, **k: p.paro_w4_experts_gated(r, fake(4, 256), *BLOCK(), **k)),
    "combine": with_routing(lambda p, r, **k: p.paro_w4_experts_combine(r, fake(8, 256), *BLOCK(), **k)),
    "gated_backward": with_routing(
        lambda p, r, **k: p.paro_w4_experts_gated_backward(r, fake(4, 256), *BLOCK(), fake(8, 32), **k)),
    "combine_backward": with_routing(
        lambda p, r, **k: p.paro_w4_experts_combine_backward(r, fake(8, 256), *BLOCK(), fake(4, 64), **k)),
    "distill": lambda p, **k: p.paro_distill_loss(fake(4, 100), fake(4, 5), fake(4, 5), **k),
}


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_memory_belongs_to_the_calls_stream(faked, monkeypatch, name):
    import torch
    monkeypatch.setattr(FakeTensor, "dtype", torch.float32, raising=False)
    s = FakeStream()
    out = STREAM_CALLS[name](faked, stream=s)
    assert FakeTensor.made and all(t.stream is s for t in FakeTensor.made)
    for t in out if isinstance(out, tuple) else (out,):
        assert t.recorded == ["current"]
    FakeTensor.made.clear()
    STREAM_CALLS[name](faked)
    assert FakeTensor.made and all(t.stream == "current" and not t.recorded for t in FakeTensor.made)


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_stream_of_another_device_is_refused(faked, monkeypatch, name):
    import torch
    monkeypatch.setattr(FakeTensor, "dtype", torch.float32, raising=False)
    s = FakeStream()
    s.device_index = 1
    with pytest.raises(ValueError, match="current device"):
        STREAM_CALLS[name](faked, stream=s)


def test_routing_and_workspace_of_another_device_are_refused(faked, monkeypatch):
    import torch
    monkeypatch.setattr(FakeTensor, "dtype", torch.float32, raising=False)
    there = fake(1 << 20)
    there.get_device = lambda: 1
    for name in STREAM_CALLS:
        if name not in ("route_backward", "distill"):
            with pytest.raises(ValueError, match="current device"):
                STREAM_CALLS[name](faked, workspace=there)
    ids = fake(4, 2)
    ids.get_device = lambda: 1
    r = faked.Routing(ids, fake(4, 2), fake(9), fake(8), fake(8))
    with pytest.raises(ValueError, match="routing"):
        faked.paro_w4_experts_gated(r, fake(4, 256), *BLOCK())
    with pytest.raises(ValueError, match="routing"):
        faked.paro_w4_experts_combine(r, fake(8, 256), *BLOCK())
