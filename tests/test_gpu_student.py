"""A student's training step, as the library's calls make it: the transform, the router, a layer of experts, the
head, the distillation loss, all their gradients and AdamW, against the derivative of the whole in fp64, and
captured."""
import numpy as np
import pytest

import oracle
import synthetic
from oracle import block, experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, H, V, TOP, G, T = 256, 384, 1040, 20, 128, 2.0


@pytest.fixture(scope="module")
def paro():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rotated_w4_linear_amd as p
    p.load_library()
    p.paro_device_init()
    return p


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


class Student:
    def __init__(self, paro, seed, M, E, k, rest):
        self.paro, self.M, self.E, self.k = paro, M, E, k
        rng = self.rng = np.random.default_rng(seed)
        _, self.layer, _ = synthetic.linear_case(seed=seed, M=1, d=D, N=16, group=G, K=4)
        self.rot = paro.Rotation(self.layer.pairs, self.layer.theta, self.layer.alpha, G)
        half = lambda *s: dev((rng.standard_normal(s) * 1.2 / np.sqrt(s[-1])).astype(np.float16))  # noqa: E731
        quantized = lambda n, d: paro.paro_quantize_weights(None, half(n, d), G)  # noqa: E731
        self.up = [t.view(E, 2 * H, -1) for t in quantized(E * 2 * H, D)]
        self.down = [t.view(E, D, -1) for t in quantized(E * D, H)]
        self.head = quantized(V, D)
        self.rest = rest
        self.scale = 64.0

    def inputs(self):
        rng, M = self.rng, self.M
        t = np.sort(rng.standard_normal((M, TOP)).astype(np.float32) * 3, 1)[:, ::-1].copy()
        index = np.stack([rng.choice(V, TOP, replace=False) for _ in range(M)]).astype(np.int32)
        lse = np.log(np.exp(t / T).sum(1) * 1.3).astype(np.float32)
        weight = rng.uniform(0.5, 1.5, M).astype(np.float32)
        if M > 2:
            weight[1] = 0.0
        return [dev(a) for a in (rng.standard_normal((M, D)).astype(np.float16),
                                 rng.standard_normal((M, self.E)).astype(np.float32), t, index, lse, weight)]

    def step(self, x, logits, t, index, lse, weight, **given):
        p = self.paro
        xr = p.paro_rotate(self.rot, x)
        r = p.paro_experts_route(logits, self.k)
        h = p.paro_w4_experts_gated(r, xr, *self.up)
        y = p.paro_w4_experts_combine(r, h, *self.down, residual=x)
        z = p.paro_w4_linear_act(None, y, *self.head)
        loss, dz = p.paro_distill_loss(z, t, index, lse=lse if self.rest else None, row_weight=weight, temperature=T,
                                       grad_scale=self.scale, dz=z)
        dy, _ = p.paro_w4_linear_act_backward(y, *self.head, dz)
        dh, dw = p.paro_w4_experts_combine_backward(r, h, *self.down, dy)
        dxr, _ = p.paro_w4_experts_gated_backward(r, xr, *self.up, dh)
        dl = p.paro_experts_route_backward(logits, r.ids, r.weights, dw, dlogits=given.get("dlogits"))
        gx, dth, dal = p.paro_rotation_backward(self.rot, x, dxr.float(), dtheta=given.get("dtheta"),
                                                dalpha=given.get("dalpha"))
        return loss, gx + dy.float(), dl, dth, dal, r.ids


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("M,E,k", [(1, 8, 2), (48, 6, 2), (300, 16, 4), (1500, 4, 1)])
def test_gradients_against_differences(paro, M, E, k, rest):
    s = Student(paro, M + rest, M, E, k, rest)
    data = s.inputs()
    print(f"student M={M} E={E} k={k} rest={rest}", flush=True)
    loss, dx, dl, dth, dal, ids = s.step(*data)
    w = [[block.weights(*(t[e].cpu().numpy() for t in q), G) for e in range(E)] for q in (s.up, s.down)]
    head = block.weights(*(t.cpu().numpy() for t in s.head), G)
    ids = ids.cpu().numpy()
    offsets, order, _ = experts.tables(ids, E)
    x, logits, t, _, lse, weight = (f64(a) for a in data)
    index = data[3].cpu().numpy()
    la = s.layer

    def total(x, logits, theta, alpha):  # the choice of the experts held
        v = oracle._apply_stages(x / alpha, la.pairs, np.cos(theta), np.sin(theta))
        e = np.exp(np.take_along_axis(logits, ids, 1))
        h, _ = experts.gated(offsets, order, k, v, w[0], None, "silu")
        y, _ = experts.combine(offsets, order, k, h, w[1], None, e / e.sum(1, keepdims=True), x)
        row = experts.distill(y @ head.T, t, index, lse if rest else None, weight, T, 1.0, "fp32")[0]
        return row.sum() * s.scale

    at = [x, logits, la.theta.astype(np.float32).astype(np.float64), la.alpha.astype(np.float32).astype(np.float64)]
    value = total(*at) / s.scale
    # h, y and z are rounded to fp16, each by at most 2^-11 of its size, and dL is at most |dz| |z| or so of that
    assert abs(f64(loss).sum() - value) < 3 * 2.0 ** -11 * (abs(value) + np.sqrt(M) * 4)
    for i, grad in enumerate((dx, dl, dth, dal)):
        if k == 1 and i == 1:  # one expert: its weight is 1, whatever its logit
            assert (f64(grad) == 0).all()
            continue
        grad = f64(grad)
        u = s.rng.standard_normal(grad.shape)
        lo, hi = list(at), list(at)
        eps = 1e-5
        lo[i], hi[i] = at[i] - eps * u, at[i] + eps * u
        num, own = (total(*hi) - total(*lo)) / (2 * eps), (grad * u).sum()
        # ten fp16 roundings of at most 2^-11 each (X', h, y, z, dz, dy, dh, the gate's and the up projection's dz,
        # dxr), at random over the elements: no more than ten times 2^-11 of the gradients' norm, which the products
        # keep, and three of that; what theta and alpha sum over the tokens, more by their number's root (it may cancel)
        size = np.linalg.norm(grad * u) if i < 2 else np.sqrt(M) * np.linalg.norm(grad * u)
        assert abs(num - own) < 32 * 2.0 ** -11 * size + 1e-5, (i, num, own, size)


@pytest.mark.parametrize("M,E,k", [(1, 8, 2), (48, 6, 2), (500, 16, 4)])
def test_captured_steps(paro, M, E, k):
    """Captured gradients with AdamW's steps between the replays, against the eager calls and steps."""
    s = Student(paro, M, M, E, k, True)
    data = [s.inputs() for _ in range(3)]
    print(f"captured student M={M} E={E} k={k}", flush=True)
    start = [s.inputs()[1], dev(s.layer.theta.astype(np.float32)), dev(s.layer.alpha.astype(np.float32))]
    runs = []
    for captured in (False, True):
        params = [a.clone() for a in start]
        grads = [torch.full_like(a, 7.0) for a in params]
        static = [a.clone() for a in data[0]]
        static[1] = params[0]  # the logits are learnt
        named = dict(zip(("dlogits", "dtheta", "dalpha"), grads))
        opt = paro.AdamW(params, grads)
        graph = None
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = s.step(*static, **named)
        seen = []
        for i in (0, 1, 2, 0):
            for j, a in enumerate(data[i]):
                if j != 1:
                    static[j].copy_(a)
            if captured:
                graph.replay()
            else:
                out = s.step(*static, **named)
            opt.step(len(seen) + 1, lr=1e-2)
            torch.cuda.synchronize()
            seen.append([a.clone() for a in (*out, *grads, *params)])
        runs.append(seen)
    for a, b in zip(*runs):
        for p, q in zip(a, b):
            assert torch.equal(p, q)
