"""The distillation loss where its numbers are at an edge: finite masks, mass that only fp64 sees; on the GPU against
the fp64 oracle, value by value, within its bounds (oracle/experts.py)."""
import numpy as np
import pytest

from oracle import experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
MASKS = {"lowest": None, "-1e30": -1e30, "-1e10": -1e10, "-65504": -65504.0}


@pytest.fixture(scope="module")
def paro():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rotated_w4_linear_amd as p
    p.load_library()
    return p


def f64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def within(got, ref, tol, what):
    assert got.shape == ref.shape, what
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - ref) <= tol) | (got == ref))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} against {ref[bad][0]}, bound {np.broadcast_to(tol, ref.shape)[bad][0]}")


def check(paro, z, values, index, lse, T, kind, what, scale=1.0):
    print(what, flush=True)
    ref = experts.distill(f64(z), f64(values), index.cpu().numpy(), None if lse is None else f64(lse), None, T, scale,
                          kind)
    assert not np.isnan(ref[0]).any() and not np.isnan(ref[2]).any() and np.isfinite(ref[3]).all(), what
    loss, dz = paro.paro_distill_loss(z, values, index, lse=lse, temperature=T, grad_scale=scale)
    within(f64(loss), ref[0], ref[1], what + " loss")
    within(f64(dz), ref[2], ref[3], what + " dz")
    over = z.clone()
    again, _ = paro.paro_distill_loss(over, values, index, lse=lse, temperature=T, grad_scale=scale, dz=over)
    torch.cuda.synchronize()
    assert torch.equal(again, loss) and torch.equal(over, dz)


def lowest(kind, mask):
    low = torch.finfo(TYPES[kind]).min
    return low if MASKS[mask] is None else max(MASKS[mask], low)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("V", [2048, 4099, 131072])
def test_finite_masks(paro, V, mask, kind, rest):
    """Masks of finite numbers, as an attention or vocabulary mask writes them: over whole lanes, at the row's start, at
    its end, over most of it, over every second logit, over an entry, over the whole row and over all but one."""
    M, K = 9, 12
    g = torch.Generator().manual_seed(V + len(mask))
    z = torch.randn((M, V), generator=g) * 2.5
    low = lowest(kind, mask)
    open_ = [slice(0, V - 548), slice(548, V), slice(V // 2, V // 2 + 40), slice(3, 60), slice(V - 40, V),
             slice(0, V, 2), slice(0, V), slice(0, 0), slice(700, 701)]
    masked = torch.full_like(z, low)
    index = torch.empty((M, K), dtype=torch.int32)
    for m, s in enumerate(open_):
        masked[m, s] = z[m, s]
        at = torch.arange(V)[s]
        pick = at[torch.randperm(len(at), generator=g)[:K]]
        index[m] = -1
        index[m, :len(pick)] = pick
    index[7, :5] = torch.tensor([0, 9, 300, 301, V - 1])
    index[6, 3] = 17
    index[6, 4:] = torch.where(index[6, 4:] == 17, -1, index[6, 4:])
    masked[6, 17] = low  # the student never takes what the teacher gives a mass
    t = torch.gather(z, 1, index.long().clamp(min=0))
    for T in (0.5, 1.0, 2.0):
        if rest:
            # (the student has mass outside the entries in every row but the last, where the teacher has none)
            full = torch.logsumexp(t.double().masked_fill(index < 0, -float("inf")) / T, 1)
            lse = (full + torch.tensor([0.25] * 8 + [-1e-3])).float().cuda()
        v = t.cuda()
        check(paro, masked.to(TYPES[kind]).cuda(), v, index.cuda(), lse if rest else None, T, kind,
              f"finite masks V={V} {mask} {kind} rest={rest} T={T}")


@pytest.mark.parametrize("shift", [1e6, -1e10, 1e20, -1e20])
def test_large_logits_differ_exactly(paro, shift):
    """Logits of which only the differences matter, however large they are: each a multiple of their spacing."""
    M, V, K = 4, 3001, 6
    g = torch.Generator().manual_seed(3)
    step = float(np.spacing(np.float32(abs(shift))))
    steps = torch.randint(-20, 1, (M, V), generator=g).double()
    z = (shift + steps * step).float()
    assert torch.equal((z.double() - shift).abs() <= 21 * step, torch.ones((M, V), dtype=torch.bool))
    index = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(M)]).int()
    values = torch.randn((M, K), generator=g)
    check(paro, z.cuda(), values.cuda(), index.cuda(), None, 2.0 * step, "fp32", f"large logits shift={shift}")


@pytest.mark.parametrize("scale", [1.0, 65536.0])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("far", [60.0, 95.0, 130.0, 300.0, 20000.0])
@pytest.mark.parametrize("V", [200, 32001])
def test_rest_far_below_the_entries(paro, V, far, kind, scale):
    """A student that is sure of the teacher's entries: its mass outside is far below what fp32 holds beside them, and
    still has a logarithm and a gradient. T takes part: far is in units of it."""
    M, K = 5, 9
    g = torch.Generator().manual_seed(V + int(far))
    z = torch.randn((M, V), generator=g)
    index = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(M)]).int()
    index[2, 4:] = -1
    index[3, 5] = index[3, 1]
    for T in (0.25, 1.0, 3.0):
        at = index.long().clamp(min=0)
        given = torch.zeros((M, V), dtype=torch.bool).scatter_(1, at, index >= 0)
        x = torch.where(given, z + far * T, z).to(TYPES[kind])
        values = torch.randn((M, K), generator=g)
        lse = torch.logsumexp(values.double().masked_fill(index < 0, -float("inf")) / T, 1)
        lse = (lse + torch.tensor([0.5, 1e-3, 0.1, 0.01, -0.1])).float().cuda()  # (the last: no rest)
        check(paro, x.cuda(), values.cuda(), index.cuda(), lse, T, kind,
              f"rest far below V={V} far={far} {kind} T={T} scale={scale}", scale)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("mask", list(MASKS))
def test_rest_masked_by_finite_numbers(paro, mask, kind):
    """All that is outside the entries masked with one large number, where the teacher has a rest: a loss of that size,
    and the rest's gradient spread over the masked logits."""
    M, V, K = 3, 5003, 7
    g = torch.Generator().manual_seed(1)
    index = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(M)]).int()
    values = torch.randn((M, K), generator=g)
    z = torch.full((M, V), lowest(kind, mask)).scatter_(1, index.long(), values + 0.1).to(TYPES[kind])
    for T in (0.5, 1.0, 2.0):
        lse = (torch.logsumexp(values.double() / T, 1) + torch.tensor([0.3, 0.01, 0.1])).float().cuda()
        check(paro, z.cuda(), values.cuda(), index.cuda(), lse, T, kind, f"rest masked {mask} {kind} T={T}")


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("V", [1, 7, 64, 2049, 40003])
def test_nan_is_never_lost(paro, V, kind, rest):
    """A logit that is NaN makes its row's loss and gradient NaN wherever it stands: alone, before anything above -inf
    that its lane reads, as a whole vector, behind masked ones, in a row that starts at any alignment."""
    rows = [slice(0, 1), slice(0, 8), slice(V - 1, V), slice(0, V), slice(V // 2, V // 2 + 1), slice(0, 16)]
    M, K = 2 * len(rows), min(5, V)
    g = torch.Generator().manual_seed(V)
    z = torch.randn((M, V), generator=g)
    index = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(M)]).int()
    values = torch.randn((M, K), generator=g)
    lse = torch.logsumexp(values, 1) + 0.1 if rest else None
    for m, s in enumerate(rows):
        z[m, s] = float("nan")
        z[m + len(rows), :V // 3] = -float("inf")
        z[m + len(rows), s] = float("nan")
    print(f"NaN V={V} {kind} rest={rest}", flush=True)
    loss, dz = paro.paro_distill_loss(z.to(TYPES[kind]).cuda(), values.cuda(), index.cuda(),
                                      lse=lse.cuda() if rest else None)
    torch.cuda.synchronize()
    assert torch.isnan(loss).all(), loss
    assert torch.isnan(dz).all(), torch.isnan(dz).all(1)
    alone, _ = paro.paro_distill_loss(z.to(TYPES[kind]).cuda(), values.cuda(), index.cuda(),
                                      lse=lse.cuda() if rest else None, gradients=False)
    assert torch.isnan(alone).all()
