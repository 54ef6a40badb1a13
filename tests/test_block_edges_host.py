"""Feed-forward products and AdamW on the CPU where arguments are at an edge: refused, or answered, before any GPU work."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def paro():
    import rotated_w4_linear_amd as p
    p.load_library()
    return p


D = ctypes.c_void_p(16 * 1024)
ODD = ctypes.c_void_p(16 * 1024 + 8)


def test_dz_without_activation_is_checked(paro):
    f = paro.load_library().paro_w4_linear_act_backward
    ws = ctypes.c_void_p(1 << 20)
    assert f(None, D, D, D, None, 0, D, ODD, D, 4, 64, 256, 128, ws, 1 << 30, None) == -5
    assert f(None, D, D, D, None, 0, D, ODD, None, 4, 64, 256, 128, None, 0, None) == -5
    assert f(None, D, D, D, None, 0, D, D, None, 4, 64, 256, 128, None, 0, None) == 0   # dz is dy: nothing to do
    assert f(None, D, D, D, None, 0, D, D, D, 4, 64, 256, 128, None, 0, None) == -7
    # nothing asked for: no workspace is looked at
    assert f(None, D, D, D, None, 0, D, None, None, 4, 64, 256, 128, ODD, 0, None) == 0


def test_backward_workspace_of_refused_sizes(paro):
    """Sizes that the calls refuse: no workspace, whatever they are, on both sides of 128 tokens."""
    import subprocess
    import sys
    # (in a process of its own: a division by zero ends it)
    code = """
import rotated_w4_linear_amd as p
lib = p.load_library()
for M in (1, 4, 128, 129, 1000, 1 << 40, (1 << 63) - 1):
    for N, d in ((64, 1), (64, 64), (64, 127), (64, 192), (17, 256), (8, 256), (1, 1), (1 << 22, 256), (64, 1 << 23)):
        for act in (0, 1):
            assert lib.paro_w4_linear_act_backward_workspace_size(M, N, d, act) == 0, (M, N, d)
        assert lib.paro_w4_gated_backward_workspace_size(M, N, d) == 0, (M, N, d)
for M in (1, 4, 128, 129):
    assert lib.paro_w4_linear_act_backward_workspace_size(M, 64, 128, 1) >= 16384
    assert lib.paro_w4_gated_backward_workspace_size(M, 64, 128) >= 16384
for M in (1 << 40, (1 << 63) - 1):
    assert lib.paro_w4_gated_backward_workspace_size(M, 64, 128) == 0
"""
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100, cwd=ROOT)
    assert res.returncode == 0, f"{res.returncode}: {res.stderr[-2000:]}"
    f = paro.load_library().paro_w4_linear_act_backward
    assert f(D, D, D, D, None, 1, D, D, D, 4, 64, 64, 64, None, 0, None) == -2


# ---------------------------------------------------------------------------
# calls on another stream: where their memory is made
# ---------------------------------------------------------------------------

class FakeTensor:
    """A device tensor as far as the wrappers look at one; notes the stream it was made on."""
    made = []
    now = "current"

    def __init__(self, shape, stream=None):
        self.shape, self.is_cuda, self.device, self.recorded = tuple(shape), True, "cuda", []
        self.stream = stream or FakeTensor.now
        if stream is None:
            FakeTensor.made.append(self)

    def new_empty(self, shape):
        return FakeTensor(shape)

    def record_stream(self, stream):
        self.recorded.append(stream)

    def data_ptr(self):
        return 0

    def is_contiguous(self):
        return True

    def numel(self):
        return 1 << 30

    def element_size(self):
        return 1

    def get_device(self):
        return 0


class FakeStream:
    device_index = 0


@pytest.fixture
def faked(paro, monkeypatch):
    """The wrappers without a GPU: allocations are noted, and no library call does anything."""
    import contextlib
    import torch

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("size") else 0

    @contextlib.contextmanager
    def on(stream):
        before, FakeTensor.now = FakeTensor.now, stream
        yield
        FakeTensor.now = before

    FakeTensor.made, FakeTensor.now = [], "current"
    make = lambda shape, *a, **k: FakeTensor((shape,) if isinstance(shape, int) else shape)  # noqa: E731
    monkeypatch.setattr(paro, "load_library", Lib)
    monkeypatch.setattr(paro, "_dptr", lambda *a: 0)
    monkeypatch.setattr(paro, "_expect", lambda *a: 0)
    monkeypatch.setattr(paro, "_stream", lambda *a: 0)
    monkeypatch.setattr(paro, "_raw_stream", lambda *a: 0)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, make)
    monkeypatch.setattr(torch, "empty_like", lambda t: FakeTensor(t.shape))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "current")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return paro


class FakePlan:
    handle, K, group = None, 8, 128


def fake(*shape):
    return FakeTensor(shape, "current")


CALLS = {
    "rotate": lambda p, **k: p.paro_rotate(FakePlan, fake(4, 256), **k),
    "quantize": lambda p, **k: p.paro_quantize_weights(None, fake(64, 256), **k),
    "linear": lambda p, **k: p.paro_w4_linear(None, fake(4, 256), fake(64, 128), fake(64, 2), fake(64, 2), **k),
    "rotation_backward": lambda p, **k: p.paro_rotation_backward(FakePlan, fake(4, 256), fake(4, 256), **k),
    "layer_loss": lambda p, **k: p.paro_layer_loss(FakePlan, fake(4, 256), fake(64, 256), fake(64, 128), fake(64, 2),
                                                   fake(64, 2), **k),
    "linear_act": lambda p, **k: p.paro_w4_linear_act(None, fake(4, 256), fake(64, 128), fake(64, 2), fake(64, 2), **k),
    "gated": lambda p, **k: p.paro_w4_gated(None, fake(4, 256), fake(64, 128), fake(64, 2), fake(64, 2), **k),
    "linear_act_backward": lambda p, **k: p.paro_w4_linear_act_backward(
        fake(4, 256), fake(64, 128), fake(64, 2), fake(64, 2), fake(4, 64), act="silu", **k),
    "gated_backward": lambda p, **k: p.paro_w4_gated_backward(
        fake(4, 256), fake(64, 128), fake(64, 2), fake(64, 2), fake(4, 32), **k),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_belongs_to_the_calls_stream(faked, name):
    """Zero-filled counters, scratch and outputs are made on the stream that the kernels run on."""
    s = FakeStream()
    out = CALLS[name](faked, stream=s)
    assert FakeTensor.made and all(t.stream is s for t in FakeTensor.made)
    # what is handed out may be used on the current stream as well
    for t in out if isinstance(out, tuple) else (out,):
        assert t is None or t.recorded == ["current"]
    FakeTensor.made.clear()
    CALLS[name](faked)
    assert FakeTensor.made and all(t.stream == "current" and not t.recorded for t in FakeTensor.made)


def test_adamw_moments_are_zero_before_any_step(faked, monkeypatch):
    """Moments made for a plan are waited for, since its steps may run on any stream; not inside a capture."""
    import torch
    log = []

    class Current:
        cuda_stream = 5

        def synchronize(self):
            log.append(("wait", len(FakeTensor.made)))

    current, capturing = Current(), [False]
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(faked, "_raw_stream", lambda s, d: s.cuda_stream if s else 5)
    monkeypatch.setattr(FakeTensor, "view", lambda self, t: self, raising=False)
    monkeypatch.setattr(FakeTensor, "dtype", torch.float32, raising=False)
    p, g = [fake(8)], [fake(8)]
    opt = faked.AdamW(p, g, state_bits=8)
    assert log == [("wait", 4)]
    other = FakeStream()
    other.cuda_stream = 6
    opt.step(1)
    assert not any(t.recorded for t in FakeTensor.made)
    opt.step(2, stream=other)
    assert all(t.recorded == [other] for t in FakeTensor.made)
    # moments of the caller's: their order is the caller's
    m, v = fake(256), fake(256)
    monkeypatch.setattr(FakeTensor, "element_size", lambda self: 4)
    opt = faked.AdamW(p, g, m, v)
    opt.step(1, stream=other)
    assert len(log) == 1 and not m.recorded
    capturing[0] = True
    with pytest.raises(ValueError, match="capture"):
        faked.AdamW(p, g)
    faked.AdamW(p, g, m, v)


def test_no_workgroup_waits_for_another(paro):
    """Workgroups that share a sum meet by counting themselves in, the last one adds: no kernel polls memory, so none
    can stay, or go on with half a sum, whatever the counters hold."""
    csrc = os.path.join(ROOT, "rotated_w4_linear_amd", "csrc")
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        for word in ("s_sleep", "__hip_atomic_load", "__nanosleep"):
            assert word not in text, f"{name}: {word}"


def test_streams_and_workspaces_of_another_device(faked, monkeypatch):
    """Refused before anything is allocated or launched."""
    other = FakeStream()
    other.device_index = 1
    for name, call in CALLS.items():
        with pytest.raises(ValueError, match="current device"):
            call(faked, stream=other)
        assert not FakeTensor.made, name
    monkeypatch.undo()
    with pytest.raises(ValueError, match="current device"):
        faked._workspace(fake(1), 0, "cuda", 1)   # a tensor on device 0
    with pytest.raises(ValueError, match="current device"):
        faked._raw_stream(FakeStream(), 1)


def test_gradients_go_where_they_are_wanted(faked):
    """Outputs that are given are the ones returned: a plan of AdamW steps reads its gradients at fixed places."""
    loss, dth, dal, gx = fake(1), fake(8, 128), fake(256), fake(4, 256)
    got = faked.paro_rotation_backward(FakePlan, fake(4, 256), fake(4, 256), gx=gx, dtheta=dth, dalpha=dal,
                                       workspace=fake(1), stream=FakeStream())
    assert got[0] is gx and got[1] is dth and got[2] is dal and not FakeTensor.made
    args = [fake(*s) for s in ((4, 256), (64, 256), (64, 128), (64, 2), (64, 2))]
    got = faked.paro_layer_loss(FakePlan, *args, loss=loss, dtheta=dth, dalpha=dal, workspace=fake(1))
    assert got[0] is loss and got[1] is dth and got[2] is dal and not FakeTensor.made
    with pytest.raises(ValueError, match="dtheta"):
        faked.paro_rotation_backward(FakePlan, fake(4, 256), fake(4, 256), dtheta=fake(8, 64))
    with pytest.raises(ValueError, match="dalpha"):
        faked.paro_layer_loss(FakePlan, *args, dalpha=fake(128))
    with pytest.raises(ValueError, match="loss"):
        faked.paro_layer_loss(FakePlan, *args, loss=fake(2))
