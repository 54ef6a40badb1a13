"""Measured cases of the mixture-of-experts operators and the distillation loss.

Operators, as a layer of experts on 4-bit weights uses them and as learning
through a whole model does:

* ``route``    softmax router: the k experts of every token, their weights, and
  the tables that put the (token, slot) pairs in expert order; ``route_grad``,
  its gradient with respect to the logits;
* ``gated``    H = act(X Wg^T + bg) * (X Wu^T + bu) of every pair by its
  expert's weights, rows in expert order; ``gated_grad``, its gradients;
* ``combine``  Y = R + sum over a token's experts of w (H W^T + b);
  ``combine_grad``, its gradients with respect to H and the weights w;
* ``distill``  T^2 KL(teacher || student) from a teacher's top logits, alone or
  with the rest of the teacher's mass as one more class, and its gradient.

A 4-bit weight stands for the fp16 number nearest to (q - z) s: that is the
format's definition, in the plain forms here as in the library.

``own`` chooses the side: the plain forms in elementary torch operations, or
the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    def route(name, op="route", **sizes):
        return {"name": name, "op": op, **sizes}

    def experts(name, op, act="silu", bias=False, residual=False, padded=0.0, group=128, **sizes):
        return {"name": name, "op": op, "act": act, "bias": bias, "residual": residual, "padded": padded,
                "group": group, **sizes}

    def distill(name, rest=False, grad=True, T=1.0, masked=0.0, **sizes):
        return {"name": name, "op": "distill", "rest": rest, "grad": grad, "T": T, "masked": masked, **sizes}

    return [
        # the router of one generated token, many small experts
        route("route 1 token", M=1, E=128, k=8, type="fp32", normalize=True, padded=0.0),
        # a long batch of prompts, a tenth of it padding, weights not normalised
        route("route 16384 tokens", M=16384, E=256, k=8, type="bf16", normalize=False, padded=0.1),
        # learning through the router, 8192 calibration tokens
        route("route grad 8192", op="route_grad", M=8192, E=64, k=6, type="fp32", normalize=True, padded=0.0),
        # one generated token through two of eight experts of a large layer
        experts("gated 1 token", "gated", M=1, E=8, k=2, d=4096, N=14336),
        # a batch of 64 sequences, one token each, over many small experts
        experts("gated 64 tokens", "gated", M=64, E=64, k=8, d=2048, N=1024),
        # a 4096-token prompt through large experts
        experts("gated 4096 tokens", "gated", M=4096, E=8, k=2, d=4096, N=14336),
        # learning through the block, 2048 calibration tokens over small experts
        experts("gated grad 2048", "gated_grad", act="gelu_tanh", bias=True, M=2048, E=32, k=4, d=2048, N=1536),
        # down projections of one generated token, added to the residual stream
        experts("combine 1 token", "combine", residual=True, M=1, E=8, k=2, d=14336, N=4096),
        # ragged: odd numbers of tokens and experts, some padding, groups of 64
        experts("combine ragged 777", "combine", bias=True, residual=True, padded=0.07, group=64, M=777, E=60, k=4,
                d=1408, N=2064),
        # learning through the down projections of large experts
        experts("combine grad 2048", "combine_grad", M=2048, E=8, k=2, d=14336, N=4096),
        # loss alone on a few rows (evaluation during learning)
        distill("distill 16 rows", grad=False, M=16, V=32000, K=32, type="bf16"),
        # a training batch, large vocabulary, the teacher's 64 top logits and the rest
        distill("distill 4096 rows", rest=True, T=2.0, masked=0.1, M=4096, V=131072, K=64, type="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "gated", "gated", "gated_grad", "combine", "combine", "combine_grad",
                     "distill", "distill"])
    if op.startswith("route"):
        E = _log_uniform(rng, 2, 256)
        return {"op": op, "M": _log_uniform(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 8)),
                "type": rng.choice(["fp32", "fp32", "fp16", "bf16"]), "normalize": rng.random() < 0.5,
                "padded": rng.choice([0.0, 0.0, 0.1, 0.5])}
    if op == "distill":
        while True:
            M, V = _log_uniform(rng, 1, 4096), _log_uniform(rng, 512, 131072)
            if M * V <= 4096 * 65536:
                break
        return {"op": op, "M": M, "V": V, "K": _log_uniform(rng, 1, 256), "rest": rng.random() < 0.5,
                "grad": rng.random() < 0.7, "T": rng.choice([1.0, 1.0, 2.0, 4.0]), "masked": rng.choice([0.0, 0.1]),
                "type": rng.choice(["fp32", "fp16", "bf16", "bf16"])}
    group = rng.choice([64, 128, 128, 256])
    step = max(128, group)
    E = _log_uniform(rng, 2, 128)
    k = rng.randint(1, min(E, 8))
    M = _log_uniform(rng, 1, 8192)
    while True:
        d = step * max(1, _log_uniform(rng, 256, 14336) // step)
        N = 16 * max(1, _log_uniform(rng, 64, 14336) // 16)
        # (the weights, and a quarter of the largest listed product: backward passes do two or three)
        if E * d * N <= 8 * 4096 * 7168 and M * k * d * N <= 2048 * 2 * 4096 * 7168:
            break
    return {"op": op, "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]), "bias": rng.random() < 0.5,
            "residual": op == "combine" and rng.random() < 0.6, "padded": rng.choice([0.0, 0.0, 0.1, 0.5]),
            "group": group, "M": M, "E": E, "k": k, "d": d, "N": N}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _quantized(gen, rows, d, group):
    """4-bit weights of N(0, 0.02): codes packed as the library stores them, fp16 scales, zeros."""
    qweight = torch.empty((rows, d // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, d // group), dtype=torch.float16, device=DEV)
    zeros = torch.empty((rows, d // group), dtype=torch.uint8, device=DEV)
    for r0 in range(0, rows, 16384):
        r1 = min(rows, r0 + 16384)
        w = torch.randn((r1 - r0, d // group, group), generator=gen, device=DEV) * 0.02
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).half()
        sf = s.float()
        z = (-lo / sf).round().clamp(0, 15)
        q = ((w / sf[..., None]).round() + z[..., None]).clamp(0, 15).to(torch.uint8).reshape(-1, d // 8, 8)
        scales[r0:r1], zeros[r0:r1] = s, z.to(torch.uint8)
        q = torch.stack([q[..., 0] | q[..., 2] << 4, q[..., 4] | q[..., 6] << 4, q[..., 1] | q[..., 3] << 4,
                         q[..., 5] | q[..., 7] << 4], -1)
        qweight[r0:r1] = q.reshape(-1, d // 2)
    return qweight, scales, zeros


def _router_logits(gen, M, E, padded):
    """Logits of a router that likes some experts better; padding tokens may use none."""
    x = torch.randn((M, E), generator=gen, device=DEV) + 0.5 * torch.randn((1, E), generator=gen, device=DEV)
    if padded:
        x[torch.rand(M, generator=gen, device=DEV) < padded] = -math.inf
    return x


def _routed(x, k, normalize):
    """ids [M][k] (-1: none), weights [M][k]: the k largest logits, the lower index first where they are equal."""
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    live = top > -math.inf
    high = x.amax(1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(top - high)
    total = e.sum(1, keepdim=True) if normalize else torch.exp(x - high).sum(1, keepdim=True)
    return torch.where(live, ids, -1).int(), torch.where(live, e / total, 0.0)


def _tables(ids, E):
    """offsets [E + 1], order (the pairs in expert order, -1 behind the last), place (the row of each pair, -1)."""
    flat = ids.flatten().long()
    key = torch.where(flat < 0, E, flat)
    order = torch.argsort(key, stable=True)
    n = (key[:, None] == torch.arange(E, device=DEV)).sum(0)
    offsets = torch.cat([n.new_zeros(1), n.cumsum(0)])
    row = torch.arange(len(flat), device=DEV)
    place = torch.empty_like(order)
    place[order] = row
    return (offsets.int(), torch.where(row < offsets[-1], order, -1).int(),
            torch.where(flat < 0, -1, place).int())


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    op, M = case["op"], case["M"]
    s = {"case": case}
    if op.startswith("route"):
        E, k = case["E"], case["k"]
        s["logits"] = _router_logits(gen, M, E, case["padded"]).to(TYPES[case["type"]])
        if op == "route_grad":  # what the forward pass has left
            s["ids"], s["weights"] = _routed(s["logits"].float(), k, case["normalize"])
            s["dweights"] = normal(M, k)
        return s
    if op == "distill":
        V, K = case["V"], case["K"]
        z = normal(M, V) * 2.5
        # the teacher: near the student, at the logits where it is large
        t = z + normal(M, V) * 0.7
        values, index = torch.topk(t, K, dim=1)
        if case["masked"]:  # rows whose teacher kept fewer logits, and tokens that the loss leaves out
            index[torch.rand((M, K), generator=gen, device=DEV) < case["masked"]] = -1
        s["z"], s["index"], s["values"] = z.to(TYPES[case["type"]]), index.int(), values.to(TYPES[case["type"]])
        s["lse"] = torch.logsumexp(t / case["T"], 1) if case["rest"] else None
        s["row_weight"] = (torch.rand(M, generator=gen, device=DEV) >= case["masked"]).float() / M
        s["scale"] = 16384.0 if case["type"] == "fp16" else 1.0  # fp16 gradients, scaled as usual
        return s
    E, k, d, N, group = case["E"], case["k"], case["d"], case["N"], case["group"]
    gated = op.startswith("gated")
    P = 2 * N if gated else N
    ids, s["weights"] = _routed(_router_logits(gen, M, E, case["padded"]), k, True)
    s["ids"] = ids
    s["offsets"], s["order"], s["place"] = _tables(ids, E)  # the router's, made once for a layer's calls
    s["qweight"], s["scales"], s["zeros"] = (t.view(E, P, -1) for t in _quantized(gen, E * P, d, group))
    s["bias"] = (normal(E, P) * 0.1).half() if case["bias"] else None
    s["residual"] = normal(M, N).half() if case["residual"] else None
    if gated:
        s["x"] = normal(M, d).half()
    else:  # rows in expert order, as the gated product leaves them
        s["h"] = (normal(M * k, d) * normal(M * k, d) * 0.5).half()
    if op == "gated":
        s["out"] = torch.zeros((M * k, N), dtype=torch.float16, device=DEV)
    elif op == "gated_grad":
        s["dh"] = normal(M * k, N).half()
        s["out"] = torch.zeros((M * k, 2 * N), dtype=torch.float16, device=DEV)
    elif op == "combine_grad":
        s["dy"] = normal(M, N).half()
        s["out"] = torch.zeros((M * k, d), dtype=torch.float16, device=DEV)
    if own:  # the router's result as its call returns it, and the workspace that a program allocates once
        import rotated_w4_linear_amd as paro
        s["routing"] = paro.Routing(ids, s["weights"], s["offsets"], s["order"], s["place"])
        new = {"combine": paro.new_experts_combine_workspace, "gated_grad": paro.new_experts_gated_backward_workspace,
               "combine_grad": paro.new_experts_combine_backward_workspace, "gated": paro.new_experts_gated_workspace}
        s["workspace"] = new[op](M, E, k, N, d)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _weights(s, hit):
    """The fp16 numbers that the codes of the experts `hit` stand for, as fp32 [experts][rows][d]."""
    group = s["case"]["group"]
    b = s["qweight"][hit]
    E, rows, half = b.shape
    b = b.view(E, rows, half // 4, 4)
    # nibbles in storage order c0 c2 c4 c6 c1 c3 c5 c7
    q = torch.stack([b & 15, b >> 4], -1).view(E, rows, half // 4, 2, 4).transpose(3, 4)
    q = q.reshape(E, rows, -1, group).float() - s["zeros"][hit].float()[..., None]
    return (q * s["scales"][hit].float()[..., None]).half().float().view(E, rows, 2 * half)


def _act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z * (z > 0)


def _act_grad(name, z):
    if name == "silu":
        t = 1 / (1 + torch.exp(-z))
        return t * (1 + z * (1 - t))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return (z > 0).to(z.dtype)


def _experts_plain(s):
    case = s["case"]
    op, M, k, N, act = case["op"], case["M"], case["k"], case["N"], case["act"]
    n = int(s["offsets"][-1])
    order = s["order"][:n].long()
    token, pair = order // k, order
    count = s["offsets"][1:] - s["offsets"][:-1]
    hit = count.nonzero().flatten()  # the experts that have rows, each padded to the longest
    count, first = count[hit], s["offsets"][hit]
    most = int(count.max()) if n else 0
    col = torch.arange(most, device=DEV)
    live = col < count[:, None]
    at = torch.where(live, first[:, None] + col, 0).long()
    expert = hit[:, None].expand(-1, most)[live]  # of each row
    w = _weights(s, hit)
    bias = s["bias"][expert].float() if s["bias"] is not None else 0.0

    def grouped(rows, transposed):  # rows in expert order, by their experts' weights
        x = rows[at] * live[..., None]
        return (torch.bmm(x, w) if transposed else torch.bmm(x, w.transpose(1, 2)))[live]

    if op.startswith("gated"):
        z = grouped(s["x"].float()[token], False) + bias
        gate, up = z[:, :N], z[:, N:]
        if op == "gated":
            s["out"][:n] = _act(act, gate) * up
            return {"h": s["out"]}
        dh = s["dh"][:n].float()
        dz = torch.cat([dh * up * _act_grad(act, gate), dh * _act(act, gate)], 1)
        s["out"][:n] = dz
        dx = torch.zeros((M * k, case["d"]), device=DEV)
        dx[pair] = grouped(dz, True)
        return {"dx": dx.view(M, k, -1).sum(1).half(), "dz": s["out"]}
    weight = s["weights"].flatten()[pair]
    if op == "combine":
        z = grouped(s["h"][:n].float(), False) + bias
        y = torch.zeros((M * k, N), device=DEV)
        y[pair] = z * weight[:, None]
        y = y.view(M, k, N).sum(1)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.half()}
    dy = s["dy"].float()[token]
    u = grouped(dy, True)
    s["out"][:n] = u * weight[:, None]
    dw = torch.zeros(M * k, device=DEV)
    dw[pair] = (u * s["h"][:n].float()).sum(1) + (dy * bias).sum(1)
    return {"dh": s["out"], "dweights": dw.view(M, k)}


def _route_plain(s):
    case = s["case"]
    x = s["logits"].float()
    if case["op"] == "route":
        ids, weights = _routed(x, case["k"], case["normalize"])
        offsets, order, place = _tables(ids, case["E"])
        return {"ids": ids, "weights": weights, "offsets": offsets, "order": order, "place": place}
    ids, w, dw = s["ids"], s["weights"], s["dweights"]
    live = ids >= 0
    inner = (w * torch.where(live, dw, 0.0)).sum(1, keepdim=True)
    if case["normalize"]:
        taken = torch.where(live, w * (dw - inner), 0.0)
        dx = torch.zeros_like(x)
    else:
        taken = torch.where(live, w * dw, 0.0)
        e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-3e38))
        dx = -inner * e / e.sum(1, keepdim=True).clamp(min=1e-30)
    dx.scatter_add_(1, ids.long().clamp(min=0), taken)
    return {"dlogits": dx.to(s["logits"].dtype)}


def _distill_plain(s):
    case = s["case"]
    T, V = case["T"], case["V"]
    x = s["z"].float() / T
    at = s["index"].long().clamp(min=0)
    t = (s["values"].double() / T).masked_fill(s["index"] < 0, -math.inf)
    if case["rest"]:
        p = torch.exp(t - s["lse"].double()[:, None])
        rest = (1 - p.sum(1)).clamp(min=0)
    else:
        p = torch.exp(t - t.amax(1, keepdim=True).clamp(min=-3e38))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    given = s["index"] >= 0
    y = s["z"].gather(1, at).double() / T - top.double()  # the student at the teacher's entries (none comes twice here)
    if case["rest"]:
        # the rest's mass by itself and the whole as its sum with the entries': where teacher and student agree,
        # the loss is a difference of nearly equal numbers
        other = torch.ones((len(x), V + 1), dtype=torch.bool, device=DEV)
        other = other.scatter_(1, torch.where(given, at, V), False)[:, :V]
        left = (e * other).sum(1, dtype=torch.float64)
        total = (left + torch.where(given, torch.exp(y), 0.0).sum(1))[:, None]
    else:
        total = e.sum(1, keepdim=True, dtype=torch.float64)
    logq = y - torch.log(total)
    live = given & (p > 0)
    loss = torch.where(live, p * (torch.log(p.clamp(min=1e-300)) - logq), 0.0).sum(1)
    if case["rest"]:
        q_rest = left / total[:, 0]
        loss = loss + torch.where(rest > 0, rest * (torch.log(rest) - torch.log(q_rest)), 0.0)
    out = {"loss": (loss * s["row_weight"] * (T * T)).float()}
    if case["grad"]:
        factor = 1 - rest / q_rest if case["rest"] else given.any(1).double()
        dz = e * (factor / total[:, 0]).float()[:, None]
        dz.scatter_add_(1, at, torch.where(given, torch.exp(logq) - p - dz.gather(1, at), 0.0).float())
        out["dz"] = (dz * (s["row_weight"] * (T * s["scale"]))[:, None]).to(s["z"].dtype)
    return out


def _run_plain(s):
    op = s["case"]["op"]
    if op.startswith("route"):
        return _route_plain(s)
    return _distill_plain(s) if op == "distill" else _experts_plain(s)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import rotated_w4_linear_amd as paro
    case = s["case"]
    op = case["op"]
    if op == "route":
        r = paro.paro_experts_route(s["logits"], case["k"], normalize=case["normalize"])
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "order": r.order, "place": r.place}
    if op == "route_grad":
        return {"dlogits": paro.paro_experts_route_backward(s["logits"], s["ids"], s["weights"], s["dweights"],
                                                            normalize=case["normalize"])}
    if op == "distill":
        loss, dz = paro.paro_distill_loss(s["z"], s["values"], s["index"], lse=s["lse"], row_weight=s["row_weight"],
                                          temperature=case["T"], grad_scale=s["scale"], gradients=case["grad"])
        return {"loss": loss} if dz is None else {"loss": loss, "dz": dz}
    weights = (s["qweight"], s["scales"], s["zeros"])
    more = {"bias": s["bias"], "group": case["group"], "workspace": s["workspace"]}
    if op == "gated":
        return {"h": paro.paro_w4_experts_gated(s["routing"], s["x"], *weights, act=case["act"], h=s["out"], **more)}
    if op == "combine":
        return {"y": paro.paro_w4_experts_combine(s["routing"], s["h"], *weights, residual=s["residual"], **more)}
    if op == "gated_grad":
        dx, dz = paro.paro_w4_experts_gated_backward(s["routing"], s["x"], *weights, s["dh"], act=case["act"],
                                                     dz=s["out"], **more)
        return {"dx": dx, "dz": dz}
    dh, dw = paro.paro_w4_experts_combine_backward(s["routing"], s["h"], *weights, s["dy"], dh=s["out"], **more)
    return {"dh": dh, "dweights": dw}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = {"fp32": 4, "fp16": 2, "bf16": 2}
    op, M = case["op"], case["M"]
    if op.startswith("route"):
        E, k = case["E"], case["k"]
        if op == "route":
            return {"bytes": M * E * size[case["type"]] + M * k * 16 + 4 * (E + 1), "flops": 4 * M * E}
        read = M * E * size[case["type"]] if not case["normalize"] else 0  # (the weights say the rest)
        return {"bytes": read + M * k * 12 + M * E * size[case["type"]], "flops": 4 * M * (k if case["normalize"] else E)}
    if op == "distill":
        V, K = case["V"], case["K"]
        z = M * V * size[case["type"]]
        return {"bytes": z * (2 if case["grad"] else 1) + M * K * (4 + size[case["type"]]) + 12 * M,
                "flops": M * V * (7 if case["grad"] else 4)}
    E, k, d, N, group = case["E"], case["k"], case["d"], case["N"], case["group"]
    live = 1 - case["padded"]
    R = M * k * live
    P = 2 * N if op.startswith("gated") else N
    # the experts that the tokens are expected to use
    hit = E * (1 - (1 - k / E) ** (M * live))
    moved = hit * (P * (d // 2) + 3 * P * (d // group) + (2 * P if case["bias"] else 0)) + 4 * R
    if op == "gated":
        return {"bytes": moved + 2 * M * live * d + 2 * R * N, "flops": 2 * R * P * d}
    if op == "gated_grad":
        return {"bytes": moved + 2 * M * live * d + 2 * R * N + 2 * R * P + 2 * M * d, "flops": 4 * R * P * d}
    if op == "combine":
        return {"bytes": moved + 2 * R * d + 2 * M * N * (2 if case["residual"] else 1) + 4 * R,
                "flops": 2 * R * N * d}
    return {"bytes": moved + 2 * M * live * N + 4 * R * d + 8 * R, "flops": 2 * R * N * d}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_experts(case, s):
    f64 = torch.float64
    op, M, k, d, N, group, name = (case[key] for key in ("op", "M", "k", "d", "N", "group", "act"))
    at = s["offsets"].tolist()
    n = at[-1]
    places = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=DEV, dtype=torch.int32)

    def weights(e):
        words = s["qweight"][e].contiguous().view(torch.int32)
        codes = ((words[:, :, None] >> places) & 15).reshape(-1, d // group, group)
        w = (codes - s["zeros"][e].int()[:, :, None]) * s["scales"][e].to(f64)[:, :, None]
        return w.half().to(f64).reshape(-1, d)

    def act(t):
        if name == "silu":
            return t * torch.sigmoid(t)
        if name == "gelu":
            return t * 0.5 * torch.erfc(-t / math.sqrt(2))
        if name == "gelu_tanh":
            return t * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))
        return t.clamp(min=0)

    def slope(t):
        if name == "silu":
            e = torch.sigmoid(t)
            return e + t * e * torch.sigmoid(-t)
        if name == "gelu":
            return 0.5 * torch.erfc(-t / math.sqrt(2)) + t * torch.exp(-t * t / 2) / math.sqrt(2 * math.pi)
        if name == "gelu_tanh":
            c = 2 * math.sqrt(2 / math.pi)
            e = torch.sigmoid(c * (t + 0.044715 * t ** 3))
            return e + t * e * (1 - e) * c * (1 + 0.134145 * t * t)
        return (t > 0).to(f64)

    R = M * k
    wide = {"gated": N, "gated_grad": 2 * N, "combine_grad": d}.get(op, 0)
    out = torch.zeros((R, wide), dtype=f64, device=DEV)
    sums = torch.zeros((M, d if op == "gated_grad" else N), dtype=f64, device=DEV)
    if s["residual"] is not None:
        sums += s["residual"].to(f64)
    dw = torch.zeros(R, dtype=f64, device=DEV)
    for e in range(case["E"]):
        a, b = at[e], at[e + 1]
        if a == b:
            continue
        pairs = s["order"][a:b].long()
        tokens = torch.div(pairs, k, rounding_mode="floor")
        w = weights(e)
        bias = s["bias"][e].to(f64) if s["bias"] is not None else torch.zeros(w.shape[0], dtype=f64, device=DEV)
        if op in ("gated", "gated_grad"):
            z = s["x"][tokens].to(f64) @ w.t() + bias
            if op == "gated":
                out[a:b] = act(z[:, :N]) * z[:, N:]
                continue
            dh = s["dh"][a:b].to(f64)
            dz = torch.cat([dh * z[:, N:] * slope(z[:, :N]), dh * act(z[:, :N])], 1)
            out[a:b] = dz
            sums.index_add_(0, tokens, dz @ w)
        elif op == "combine":
            share = s["weights"].flatten()[pairs].to(f64)[:, None]
            sums.index_add_(0, tokens, share * (s["h"][a:b].to(f64) @ w.t() + bias))
        else:
            dy = s["dy"][tokens].to(f64)
            u = dy @ w
            out[a:b] = u * s["weights"].flatten()[pairs].to(f64)[:, None]
            dw[pairs] = (u * s["h"][a:b].to(f64)).sum(1) + dy @ bias
    if op == "gated":
        return {"h": out}
    if op == "gated_grad":
        return {"dx": sums, "dz": out}
    return {"y": sums} if op == "combine" else {"dh": out, "dweights": dw.view(M, k)}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op == "route":
        x = s["logits"].to(f64)
        ids, _ = _routed(x, case["k"], case["normalize"])
        p = torch.softmax(x.clamp(min=-1e300), 1) * (x > -math.inf)
        w = p.gather(1, ids.long().clamp(min=0)) * (ids >= 0)
        if case["normalize"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        return {"ids": None, "weights": w, "offsets": None, "order": None, "place": None}
    if op == "route_grad":
        x = s["logits"].to(f64).clone().requires_grad_()
        taken = torch.zeros_like(x).scatter_add_(1, s["ids"].long().clamp(min=0), (s["ids"] >= 0).to(f64)) > 0
        full = ~taken.any(1)
        kept = x.masked_fill(~taken, -math.inf) if case["normalize"] else x
        p = torch.softmax(kept.masked_fill(full[:, None], 0.0), 1)
        up = torch.zeros_like(x).scatter_add_(1, s["ids"].long().clamp(min=0),
                                              torch.where(s["ids"] >= 0, s["dweights"], 0.0).to(f64))
        (p * up).sum().backward()
        return {"dlogits": torch.nan_to_num(x.grad, nan=0.0)}
    if op == "distill":
        T, V, M = case["T"], case["V"], case["M"]
        losses, grads = [], []
        for a in range(0, M, 512):
            z = s["z"][a:a + 512].to(f64)
            index, value = s["index"][a:a + 512].long(), s["values"][a:a + 512].to(f64)
            target = torch.zeros_like(z)
            kept = torch.zeros_like(z)
            live = (index >= 0).to(f64)
            kept.scatter_add_(1, index.clamp(min=0), live)
            if case["rest"]:
                p = torch.exp(value / T - s["lse"][a:a + 512].to(f64)[:, None]) * live
            else:
                p = torch.softmax((value / T).masked_fill(live == 0, -1e300), 1) * live
            target.scatter_add_(1, index.clamp(min=0), p)
            logq = torch.log_softmax(z / T, 1)
            loss = (torch.xlogy(target, target) - target * logq).sum(1)
            dz = torch.exp(logq) * target.sum(1, keepdim=True) - target
            if case["rest"]:
                left = (1 - target.sum(1)).clamp(min=0)
                outside = logq.masked_fill(kept > 0, -math.inf)
                lse_out = torch.logsumexp(outside, 1)
                loss = loss + torch.xlogy(left, left) - torch.where(left > 0, left * lse_out, 0.0)
                dz = dz + left[:, None] * (torch.exp(logq) - torch.exp(outside - lse_out[:, None]))
            share = s["row_weight"][a:a + 512].to(f64)
            losses.append(loss * share * T * T)
            if case["grad"]:
                grads.append(dz * (share * T * s["scale"])[:, None])
        out = {"loss": torch.cat(losses)}
        return out | {"dz": torch.cat(grads)} if case["grad"] else out
    return _exact_experts(case, s)
