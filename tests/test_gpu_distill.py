"""The distillation loss on the GPU against the fp64 oracle, value by value, within the
bounds that follow from the documented arithmetic (oracle/experts.py)."""
import numpy as np
import pytest

from oracle import experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def paro():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rotated_w4_linear_amd as p
    p.load_library()
    return p


def log(msg):
    print(msg, flush=True)


def f64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def within(got, ref, tol, what):
    assert got.shape == ref.shape, what
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - ref) <= tol) | (np.isnan(ref) & np.isnan(got)) | (got == ref))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} against {ref[bad][0]}, bound {np.broadcast_to(tol, ref.shape)[bad][0]}")


def inputs(seed, M, V, K, kind, tkind, T, near=0.7):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((M, V), generator=g) * 2.5
    t = z + near * torch.randn((M, V), generator=g)
    values, index = torch.topk(t, K, dim=1)
    lse = torch.logsumexp(t.double() / T, 1).float()
    return z.to(TYPES[kind]).cuda(), values.to(TYPES[tkind]).cuda(), index.int().cuda(), lse.cuda()


def check(paro, z, values, index, lse, w, T, scale, kind, what):
    log(what)
    zh = f64(z)
    guard = torch.full((z.numel() + 64,), 7.0, dtype=z.dtype, device="cuda")
    dz = guard[32:-32].view(z.shape)
    loss, got = paro.paro_distill_loss(z, values, index, lse=lse, row_weight=w, temperature=T, grad_scale=scale, dz=dz)
    ref = experts.distill(zh, f64(values), index.cpu().numpy(), None if lse is None else f64(lse),
                          None if w is None else f64(w), T, scale, kind)
    within(f64(loss), ref[0], ref[1], what + " loss")
    within(f64(got), ref[2], ref[3], what + " dz")
    assert (guard[:32] == 7).all() and (guard[-32:] == 7).all(), "written outside the output"
    # the loss alone, and the gradient over the logits
    alone, none = paro.paro_distill_loss(z, values, index, lse=lse, row_weight=w, temperature=T, gradients=False)
    assert none is None and torch.equal(alone.view(torch.int32), loss.view(torch.int32))
    over = z.clone()
    paro.paro_distill_loss(over, values, index, lse=lse, row_weight=w, temperature=T, grad_scale=scale, dz=over)
    torch.cuda.synchronize()
    bits = torch.int32 if z.element_size() == 4 else torch.int16
    assert torch.equal(over.view(bits), got.view(bits))


# rows that start at any alignment (odd V), fewer logits than lanes, one logit, as many
# entries as logits, and beyond what stays in registers
SIZES = [(1, 1, 1), (2, 2, 1), (3, 7, 7), (5, 63, 3), (2, 255, 64), (4, 513, 20), (3, 1000, 1000), (7, 4099, 33),
         (2, 32001, 256), (3, 50000, 64), (1, 65537, 1024), (2, 131072, 64), (2, 131077, 10), (1, 262147, 100),
         (1, 1 << 20, 7)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M,V,K", SIZES)
def test_distill(paro, M, V, K, kind):
    for i, (T, tkind) in enumerate([(1.0, "fp32"), (2.0, kind)]):
        z, values, index, lse = inputs(V + K + i, M, V, K, kind, tkind, T)
        scale = 256.0 if kind == "fp16" else 1.0
        w = torch.linspace(0.5, 2.0, M).cuda()
        check(paro, z, values, index, None, w, T, scale, kind, f"distill M={M} V={V} K={K} {kind} T={T}")
        check(paro, z, values, index, lse, None, T, scale, kind, f"distill rest M={M} V={V} K={K} {kind} T={T}")


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
def test_masks(paro, kind, rest):
    """Rows left out (NaN in them), rows without entries, entries out of range, masked entries, masked student logits,
    an index that comes twice and more often."""
    M, V, K, T = 12, 3001, 40, 1.5
    z, values, index, lse = inputs(5, M, V, K, kind, "fp32", T)
    w = torch.ones(M, device="cuda")
    w[1] = 0.0
    z[1, 5], values[1, 3] = float("nan"), float("nan")
    index[2] = -1
    index[3, ::2], index[3, 1] = -5, V
    index[4, 7], index[4, 9] = 2 ** 31 - 1, -2 ** 31
    values[5, 3:] = -float("inf")
    values[6] = -float("inf")
    z[7, 1000:2000] = -float("inf")
    index[7] = torch.arange(K, device="cuda", dtype=torch.int32) * 7
    z[7, ::7][:K] = 1.0
    index[8, 1:] = index[8, 0]
    index[9, 11] = index[9, 3]
    index[9, 30] = index[9, 3]
    values[10, 4] = -float("inf")
    z[10, int(index[10, 4])] = -float("inf")
    z[11, 17:] = -float("inf")
    index[11] = -1
    index[11, :3] = torch.tensor([0, 3, 16])
    check(paro, z, values, index, lse if rest else None, w, T, 64.0, kind, f"masks {kind} rest={rest}")


def test_student_without_mass_outside_the_entries(paro):
    z = torch.full((2, 64), -float("inf"), device="cuda")
    z[:, :4] = torch.tensor([1.0, 2.0, 0.5, -1.0])
    index = torch.arange(4, dtype=torch.int32, device="cuda").repeat(2, 1)
    values = z[:, :4].contiguous()
    lse = torch.logsumexp(values, 1)
    lse[1] += 0.5  # the teacher has a rest, the student none: an infinite loss
    log("no mass outside")
    loss, dz = paro.paro_distill_loss(z, values, index, lse=lse)
    torch.cuda.synchronize()
    assert abs(loss[0].item()) < 1e-6 and loss[1].item() == float("inf")
    assert torch.isfinite(dz).all() and not dz[:, 4:].any()


@pytest.mark.parametrize("kind", list(TYPES))
def test_not_finite_stays_in_its_row(paro, kind):
    M, V, K = 6, 5000, 16
    z, values, index, lse = inputs(11, M, V, K, kind, "fp32", 1.0)
    for l in (None, lse):
        log(f"not finite {kind} rest={l is not None}")
        loss, dz = paro.paro_distill_loss(z, values, index, lse=l)
        bad = z.clone()
        bad[1, 100], bad[2, 4999], bad[3, 0] = float("nan"), float("inf"), float("nan")
        lost, dbad = paro.paro_distill_loss(bad, values, index, lse=l)
        torch.cuda.synchronize()
        keep = [0, 4, 5]
        assert torch.equal(lost[keep], loss[keep]) and torch.equal(dbad[keep], dz[keep])
        assert torch.isnan(lost[1:4]).all()


def test_far_from_the_teacher(paro):
    """Large logits, far apart: no overflow, and the small differences kept."""
    M, V, K = 3, 2000, 8
    z, values, index, lse = inputs(13, M, V, K, "fp32", "fp32", 1.0)
    for factor, shift in ((30.0, 0.0), (1.0, 1e4), (1e-3, -300.0)):
        check(paro, z * factor + shift, values * factor + shift, index, None, None, 1.0, 1.0, "fp32",
              f"far factor={factor} shift={shift}")


def test_captured_and_on_another_stream(paro):
    M, V, K = 5, 9001, 12
    data = [inputs(s, M, V, K, "bf16", "bf16", 1.0) for s in range(3)]
    want = [paro.paro_distill_loss(*d[:3], lse=d[3]) for d in data]
    static = [t.clone() for t in data[0]]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        paro.paro_distill_loss(*static[:3], lse=static[3])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = paro.paro_distill_loss(*static[:3], lse=static[3])
    for i in (1, 2, 0, 1):
        for s, d in zip(static, data[i]):
            s.copy_(d)
        g.replay()
        got = paro.paro_distill_loss(*data[i][:3], lse=data[i][3], stream=side)
        torch.cuda.synchronize()
        for a, b, c in zip(out, want[i], got):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_largest(paro):
    """More than 2^31 logits, as many in a row as there can be, with as many of the teacher's; some rows compared."""
    M, V, K, T = 2100, 1 << 20, 1024, 1.5
    print("distill largest", flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.empty((M, V), dtype=torch.float16, device="cuda").normal_(0, 2.5, generator=g)
    values = torch.randn((M, K), device="cuda", generator=g) * 4
    index = (torch.randperm(V, device="cuda", generator=g)[:K] - torch.arange(M, device="cuda")[:, None]) % V
    index = index.int()
    lse = torch.logsumexp(values / T, 1) + 0.1
    loss, dz = paro.paro_distill_loss(z, values, index, lse=lse, temperature=T, grad_scale=1000.0)
    at = torch.tensor([0, 2046, 2047, 2048, M - 1], device="cuda")
    ref = experts.distill(f64(z[at]), f64(values[at]), index[at].cpu().numpy(), f64(lse[at]), None, T, 1000.0, "fp16")
    within(f64(loss[at]), ref[0], ref[1], "loss")
    within(f64(dz[at]), ref[2], ref[3], "dz")


def test_python_refusals(paro):
    z, values, index, lse = inputs(1, 4, 100, 8, "fp32", "fp32", 1.0)
    with pytest.raises(TypeError):
        paro.paro_distill_loss(z.double(), values, index)
    with pytest.raises(TypeError):
        paro.paro_distill_loss(z, values, index.long())
    with pytest.raises(ValueError):
        paro.paro_distill_loss(z, values, index[:3])
    with pytest.raises(ValueError):
        paro.paro_distill_loss(z[:, ::2], values, index)
    with pytest.raises(paro.ParoError):
        paro.paro_distill_loss(z, values, index, temperature=0.0)
    with pytest.raises(TypeError):
        paro.paro_distill_loss(z, values, index, dz=torch.empty_like(z, dtype=torch.float16))
    loss, dz = paro.paro_distill_loss(z[:0], values[:0], index[:0])
    assert loss.shape == (0,) and dz.shape == (0, 100)
