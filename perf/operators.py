"""Measured cases of the feed-forward and learning operators of the library.

Three operators, as the feed-forward half of a decoder layer uses them:

* ``linear``  Y = act(X W^T + b) + R on 4-bit weights (bias, activation and
  residual in the product's epilogue), and ``linear_grad``, its gradients with
  respect to the pre-activation and the input;
* ``gated``   Y = act(X Wg^T + bg) * (X Wu^T + bu) on 4-bit weights stored as
  one [2N] block (gate rows, then up rows), and ``gated_grad``, its gradients;
* ``adamw``   one AdamW step over many tensors, moments in 32 bits or in 8
  (e4m3 values with one fp32 scale per block of 256).

X is what the product multiplies: activations that are transformed already.
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
BLOCK = 256            # moments that share a scale in the 8-bit form
E4M3_MAX = 448.0
TINY = 2.0 ** -100     # a block whose largest moment is below this is held as zero
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.01, 100

# in_features and out_features of the linears of a Llama-3-8B decoder layer
LAYER = [(4096, 4096), (4096, 1024), (4096, 1024), (4096, 4096), (4096, 14336), (4096, 14336),
         (14336, 4096)]


def listed():
    def linear(name, op="linear", act="none", bias=False, residual=False, **sizes):
        return {"name": name, "op": op, "act": act, "bias": bias, "residual": residual, **sizes}

    def adamw(name, tensors, param, grad, bits, layers=0):
        return {"name": name, "op": "adamw", "tensors": tensors, "layers": layers, "param": param, "grad": grad,
                "bits": bits}

    return [
        # attention output projection of one generated token, added to the residual stream
        linear("o_proj 1 token", residual=True, M=1, d=4096, N=4096, group=128),
        # down projection of a batch of 16 sequences, one token each
        linear("down 16 tokens", bias=True, residual=True, M=16, d=14336, N=4096, group=128),
        # down projection of a 2048-token prompt
        linear("down 2048 tokens", residual=True, M=2048, d=14336, N=4096, group=128),
        # an ungated feed-forward layer with bias, ragged batch, odd width, groups of 64
        linear("ragged 333 gelu", act="gelu", bias=True, residual=True, M=333, d=2560, N=1040, group=64),
        # learning through a layer with bias and activation, 1024 calibration tokens
        linear("grad 1024 gelu_tanh", op="linear_grad", act="gelu_tanh", bias=True, M=1024, d=4096, N=4096,
               group=128),
        # gate and up projections of one generated token
        linear("gated 1 token", op="gated", act="silu", M=1, d=4096, N=14336, group=128),
        # the same of a 2048-token prompt
        linear("gated 2048 tokens", op="gated", act="silu", M=2048, d=4096, N=14336, group=128),
        # an 8K-token prompt: the largest product
        linear("gated 8192 tokens", op="gated", act="silu", M=8192, d=4096, N=14336, group=128),
        # learning through the block, 2048 calibration tokens
        linear("gated grad 2048", op="gated_grad", act="silu", M=2048, d=4096, N=14336, group=128),
        # angles and scales of one decoder layer (14 tensors), 8-bit moments: launch latency
        adamw("adamw layer angles 8-bit", "angles", "fp32", "fp32", 8, layers=1),
        # angles and scales of 32 decoder layers (448 tensors), 32-bit moments
        adamw("adamw model angles", "angles", "fp32", "fp32", 32, layers=32),
        # the weights of one decoder layer, gradients in fp16, 8-bit moments
        adamw("adamw layer weights 8-bit", "weights", "fp32", "fp16", 8, layers=1),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "gated", "gated", "gated_grad", "adamw", "adamw"])
    if op == "adamw":
        # an odd-sized tensor list: the sizes follow from the seed and the total
        return {"op": op, "tensors": "random", "layers": 0, "count": _log_uniform(rng, 1, 600),
                "total": _log_uniform(rng, 1000, 60_000_000), "sizes_seed": rng.randrange(1 << 30),
                "param": rng.choice(["fp32", "fp32", "fp16", "bf16"]), "grad": rng.choice(["fp32", "fp16", "bf16"]),
                "bits": rng.choice([32, 8])}
    group = rng.choice([64, 128, 128, 256])
    step = max(128, group)
    M = _log_uniform(rng, 1, 8192)
    while True:
        d = step * max(1, _log_uniform(rng, 128, 14336) // step)
        N = 16 * max(1, _log_uniform(rng, 32, 14336) // 16)
        if M * N * d <= 8192 * 4096 * 7168:  # (backward passes do twice the products)
            break
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"] + ([] if op.startswith("gated") else ["none"]))
    return {"op": op, "act": act, "bias": rng.random() < 0.5,
            "residual": op == "linear" and rng.random() < 0.6, "M": M, "d": d, "N": N, "group": group}


def _sizes(case):
    """Tensor sizes of an adamw case."""
    if case["tensors"] == "angles":  # theta [8][d / 2] and alpha [d] of every linear
        return [n for _ in range(case["layers"]) for d, _ in LAYER for n in (4 * d, d)]
    if case["tensors"] == "weights":
        return [d * N for d, N in LAYER] * case["layers"]
    import random
    rng = random.Random(case["sizes_seed"])
    parts = [rng.random() ** 3 + 1e-4 for _ in range(case["count"])]
    return [max(1, int(case["total"] * p / sum(parts))) for p in parts]


TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def _quantized(gen, rows, d, group):
    """4-bit weights of N(0, 0.02): codes packed as the library stores them, fp16 scales, zeros."""
    qweight = torch.empty((rows, d // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, d // group), dtype=torch.float16, device=DEV)
    zeros = torch.empty((rows, d // group), dtype=torch.uint8, device=DEV)
    for r0 in range(0, rows, 8192):
        r1 = min(rows, r0 + 8192)
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


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "adamw":
        sizes = _sizes(case)
        padded = [-(-n // BLOCK) * BLOCK for n in sizes]
        total = sum(padded)
        # parameters and gradients as views of one buffer each, every tensor
        # from a multiple of 256 values on (as gradient buckets are laid out);
        # the padding between them is zero and stays so
        keep = torch.zeros(total, dtype=torch.bool, device=DEV)
        starts = [0]
        for n, p in zip(sizes, padded):
            keep[starts[-1]:starts[-1] + n] = True
            starts.append(starts[-1] + p)
        p = torch.randn(total, generator=gen, device=DEV) * 0.5 * keep
        # gradients of very different size from tensor to tensor and inside one
        g = torch.randn(total, generator=gen, device=DEV) * 0.01 * keep
        g *= torch.randn(total, generator=gen, device=DEV).abs()
        m = torch.randn(total, generator=gen, device=DEV) * 0.003 * keep
        v = (torch.randn(total, generator=gen, device=DEV) * 0.01 * keep).square()
        s["p"], s["g"] = p.to(TYPES[case["param"]]), g.to(TYPES[case["grad"]])
        if case["bits"] == 32:
            s["m"], s["v"], s["ms"], s["vs"] = m, v, None, None
        else:
            s["m"], s["ms"] = _to8(m, torch.ones_like(keep[:1]))
            s["v"], s["vs"] = _to8(v.sqrt(), v > 0)
        del p, g, m, v, keep
        if own:  # the plan of tensors that a training loop makes once
            import rotated_w4_linear_amd as paro
            cut = lambda t: [t[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
            s["plan"] = paro.AdamW(cut(s["p"]), cut(s["g"]), s["m"], s["v"], s["ms"], s["vs"])
        return s
    M, d, N, group = case["M"], case["d"], case["N"], case["group"]
    rows = 2 * N if op.startswith("gated") else N
    x = torch.randn((M, d), generator=gen, device=DEV)
    # (the transform's purpose: rotated activations have mild outliers only)
    s["x"] = x.half()
    s["qweight"], s["scales"], s["zeros"] = _quantized(gen, rows, d, group)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s["bias"] = (normal(rows) * 0.1).half() if case["bias"] else None
    s["residual"] = normal(M, N).half() if case["residual"] else None
    if op.endswith("_grad"):
        s["dy"] = normal(M, N).half()
    if own:  # the workspace that a serving or training loop allocates once
        import rotated_w4_linear_amd as paro
        s["workspace"] = {
            "linear": lambda: paro.new_workspace(None, M, N, d),
            "linear_grad": lambda: paro.new_linear_act_backward_workspace(M, N, d, case["act"]),
            "gated": lambda: paro.new_gated_workspace(None, M, N, d),
            "gated_grad": lambda: paro.new_gated_backward_workspace(M, N, d),
        }[op]()
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _weights(s):
    """The fp16 numbers that the codes stand for, as fp32 [rows][d]."""
    group = s["case"]["group"]
    b = s["qweight"]
    rows, half = b.shape
    b = b.view(rows, half // 4, 4)
    # nibbles in storage order c0 c2 c4 c6 c1 c3 c5 c7
    q = torch.stack([b & 15, b >> 4], -1).view(rows, half // 4, 2, 4).transpose(2, 3)
    q = q.reshape(rows, -1, group).float() - s["zeros"].float()[..., None]
    return (q * s["scales"].float()[..., None]).half().float().view(rows, 2 * half)


def _act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "relu":
        return z * (z > 0)
    return z


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
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def _to8(x, positive):
    """x as e4m3 values of its block's largest magnitude / 448; nonzero where `positive`."""
    top = x.view(-1, BLOCK).abs().amax(1)
    top = top * (top >= TINY)
    inv = torch.where(top > 0, E4M3_MAX / top, top)
    code = (x.view(-1, BLOCK) * inv[:, None]).view(-1).to(torch.float8_e4m3fn)
    if positive.numel() == x.numel():  # second moments: the smallest value instead of zero
        bits = code.view(torch.uint8)
        live = positive & (top > 0).repeat_interleave(BLOCK)
        code = torch.maximum(bits, live.to(torch.uint8)).view(torch.float8_e4m3fn)
    return code, top / E4M3_MAX


def _adamw_plain(s):
    eight = s["case"]["bits"] == 8
    g, p = s["g"].float(), s["p"].float()
    if eight:
        m = (s["m"].float().view(-1, BLOCK) * s["ms"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["vs"][:, None]).view(-1)
        v = v * v
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = torch.sqrt(v)
    c1, c2 = 1 - BETA1 ** STEP, math.sqrt(1 - BETA2 ** STEP)
    p = p * (1 - LR * DECAY) - (m / (root / c2 + EPS)) * (LR / c1)
    s["p"].copy_(p)
    if eight:
        for key, scale, value, positive in (("m", "ms", m, m[:1] > 0), ("v", "vs", root, v > 0)):
            code, top = _to8(value, positive)
            s[key].copy_(code)
            s[scale].copy_(top)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "adamw":
        _adamw_plain(s)
        return _adamw_out(s)
    N, act = case["N"], case["act"]
    w = _weights(s)
    x = s["x"].float()
    if op == "linear_grad" and act == "none":
        return {"dx": (s["dy"].float() @ w).half()}
    z = x @ w.T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if op == "linear":
        z = _act(act, z)
        if s["residual"] is not None:
            z = z + s["residual"].float()
        return {"y": z.half()}
    if op == "gated":
        return {"y": (_act(act, z[:, :N]) * z[:, N:]).half()}
    dy = s["dy"].float()
    if op == "linear_grad":
        dz = dy * _act_grad(act, z)
    else:
        gate, up = z[:, :N], z[:, N:]
        dz = torch.cat([dy * up * _act_grad(act, gate), dy * _act(act, gate)], 1)
    return {"dx": (dz @ w).half(), "dz": dz.half()}


def _adamw_out(s):
    out = {"p": s["p"], "m": s["m"], "v": s["v"]}
    if s["ms"] is not None:
        out |= {"ms": s["ms"], "vs": s["vs"]}
    return out


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import rotated_w4_linear_amd as paro
    case = s["case"]
    op = case["op"]
    if op == "adamw":
        s["plan"].step(STEP, lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY)
        return _adamw_out(s)
    weights = (s["qweight"], s["scales"], s["zeros"])
    more = {"act": case["act"], "group": case["group"], "workspace": s["workspace"]}
    if op == "linear":
        return {"y": paro.paro_w4_linear_act(None, s["x"], *weights, bias=s["bias"], residual=s["residual"], **more)}
    if op == "gated":
        return {"y": paro.paro_w4_gated(None, s["x"], *weights, bias=s["bias"], **more)}
    back = paro.paro_w4_linear_act_backward if op == "linear_grad" else paro.paro_w4_gated_backward
    dx, dz = back(s["x"], *weights, s["dy"], bias=s["bias"], **more)
    return {"dx": dx} if dz is None else {"dx": dx, "dz": dz}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        size = {"fp32": 4, "fp16": 2, "bf16": 2}
        moments = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * (2 * size[case["param"]] + size[case["grad"]] + moments), "flops": 14 * n}
    M, d, N, op = case["M"], case["d"], case["N"], case["op"]
    rows = 2 * N if op.startswith("gated") else N
    weights = rows * (d // 2) + 3 * rows * (d // case["group"])
    acted = op.startswith("gated") or case["act"] != "none"
    if op in ("linear", "gated"):
        moved = weights + 2 * M * d + 2 * M * N * (2 if case["residual"] else 1)
        return {"bytes": moved + (2 * rows if case["bias"] else 0), "flops": 2 * M * rows * d}
    if not acted:
        return {"bytes": weights + 2 * M * N + 2 * M * d, "flops": 2 * M * N * d}
    moved = weights + 2 * M * d + 2 * M * N + 2 * M * rows + 2 * M * d + (2 * rows if case["bias"] else 0)
    return {"bytes": moved, "flops": 4 * M * rows * d}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "adamw":
        p, g = s["p"].to(f64), s["g"].to(f64)
        eight = case["bits"] == 8
        m, v = s["m"].to(f64), s["v"].to(f64)
        if eight:
            m = m * s["ms"].to(f64).repeat_interleave(BLOCK)
            v = (v * s["vs"].to(f64).repeat_interleave(BLOCK)) ** 2
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        mhat, vhat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        out = {"p": p - LR * DECAY * p - LR * mhat / (vhat.sqrt() + EPS)}
        if not eight:
            return out | {"m": m, "v": v}
        for key, scale, value in (("m", "ms", m), ("v", "vs", v.sqrt())):
            top = value.reshape(-1, BLOCK).abs().max(1).values
            top = torch.where(top < TINY, torch.zeros_like(top), top)
            out[scale] = top / 448
            unit = (top / 448).repeat_interleave(BLOCK)
            live = unit > 0
            code = torch.where(live, value / torch.where(live, unit, torch.ones_like(unit)), torch.zeros_like(value))
            code = code.to(torch.float8_e4m3fn).to(f64)
            if key == "v":
                code = torch.where(live & (v > 0), code.clamp(min=2.0 ** -9), code)
            out[key] = code
        return out
    N, d, group = case["N"], case["d"], case["group"]
    words = s["qweight"].contiguous().view(torch.int32)
    places = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=DEV, dtype=torch.int32)
    codes = ((words[:, :, None] >> places) & 15).reshape(-1, d // group, group)
    w = ((codes - s["zeros"].int()[:, :, None]) * s["scales"].to(f64)[:, :, None]).half().to(f64).reshape(-1, d)
    del words, codes
    z = torch.matmul(s["x"].to(f64), w.t())
    if s["bias"] is not None:
        z += s["bias"].to(f64)
    name = case["act"]
    root = 1 / math.sqrt(2)

    def act(t):
        if name == "silu":
            return t * torch.sigmoid(t)
        if name == "gelu":
            return t * 0.5 * torch.erfc(-t * root)
        if name == "gelu_tanh":
            return t * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))
        return t.clamp(min=0) if name == "relu" else t

    def slope(t):
        if name == "silu":
            e = torch.sigmoid(t)
            return e + t * e * torch.sigmoid(-t)
        if name == "gelu":
            return 0.5 * torch.erfc(-t * root) + t * torch.exp(-t * t / 2) * root / math.sqrt(math.pi)
        if name == "gelu_tanh":
            c = 2 * math.sqrt(2 / math.pi)
            e = torch.sigmoid(c * (t + 0.044715 * t ** 3))
            return e + t * e * (1 - e) * c * (1 + 0.134145 * t * t)
        return (t > 0).to(f64) if name == "relu" else torch.ones_like(t)

    op = case["op"]
    if op == "linear":
        y = act(z)
        return {"y": y if s["residual"] is None else y + s["residual"].to(f64)}
    if op == "gated":
        return {"y": act(z[:, :N]) * z[:, N:]}
    dy = s["dy"].to(f64)
    if op == "linear_grad":
        dz = dy * slope(z)
        return {"dx": dz @ w} if name == "none" else {"dx": dz @ w, "dz": dz}
    dz = torch.cat([dy * z[:, N:] * slope(z[:, :N]), dy * act(z[:, :N])], dim=1)
    return {"dx": dz @ w, "dz": dz}
