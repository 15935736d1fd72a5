"""Cases of the layer operators: the linear product with its epilogue and its
gradients, the per-head norms of queries and keys with the position rotation
in the same pass, and the rotation by positions with several axes.

`run` computes each in its plain form (elementary torch operations in fp32,
angles in fp64, one rounding at the end) or, with `own` set, through this
package's entry points.  `exact` gives the same results in fp64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # One token through a fused q/k/v projection (32 query, 8 key and 8 value heads of 128): serving latency,
        # bound by reading the weight.
        dict(name="linear decode 1 token", op="linear", m=1, k=4096, n=6144, dtype="bf16", act="none",
             bias=True, residual="none", save=False),
        # 48 sequences decoding together through the first MLP matrix.
        dict(name="linear decode 48 tokens", op="linear", m=48, k=4096, n=14336, dtype="bf16", act="silu",
             bias=False, residual="none", save=False),
        # Training forward of the first MLP matrix of a Llama-3-8B-shaped layer, pre-activation kept for backward.
        dict(name="linear train up", op="linear", m=4096, k=4096, n=14336, dtype="bf16", act="gelu_tanh",
             bias=True, residual="none", save=True),
        # A ragged prompt through a small model's second MLP matrix with odd widths, onto an fp32 residual stream.
        dict(name="linear odd prompt", op="linear", m=1037, k=2050, n=1001, dtype="bf16", act="silu",
             bias=True, residual="f32", save=False),
        # Gradients of the first MLP matrix: input, weight and bias.
        dict(name="linear backward up", op="linear_backward", m=4096, k=4096, n=14336, dtype="bf16", act="gelu_tanh",
             bias=True, dw="bf16"),
        # Gradients of the fused q/k/v projection, the weight's in fp32 as the optimizer step takes it.
        dict(name="linear backward qkv", op="linear_backward", m=2048, k=4096, n=6144, dtype="bf16", act="none",
             bias=False, dw="f32"),
        # A small fp32 layer, as the fp32 mode of the step serves.
        dict(name="linear backward fp32", op="linear_backward", m=509, k=768, n=1024, dtype="f32", act="gelu",
             bias=True, dw="f32"),
        # 16 sequences decoding, 32 query and 8 key heads, one position each.
        dict(name="qk norm decode", op="qk", tokens=16, hq=32, hk=8, dim=128, dtype="bf16", rot=128,
             interleaved=False, backward=False, far=100000),
        # A training batch of 8192 tokens, q and k read as views of the packed q/k/v rows.
        dict(name="qk norm train", op="qk", tokens=8192, hq=32, hk=8, dim=128, dtype="bf16", rot=128,
             interleaved=False, backward=False, far=8192),
        # Its gradients: q, k and both norm weights.
        dict(name="qk norm train backward", op="qk", tokens=8192, hq=32, hk=8, dim=128, dtype="bf16", rot=128,
             interleaved=False, backward=True, far=8192),
        # A long image and video prompt: time, height and width positions over 16, 24 and 24 of the 64 pairs.
        dict(name="rope 3 axes prompt", op="rope", tokens=30011, hq=28, hk=4, dim=128, dtype="bf16", axes=3,
             rot=128, interleaved=False, backward=False, far=30000),
        # Gradients of a vision tower's rotation over rows and columns, fp32, heads of 80.
        dict(name="rope 2 axes backward", op="rope", tokens=1531, hq=16, hk=16, dim=80, dtype="f32", axes=2,
             rot=80, interleaved=True, backward=True, far=4096),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size spread over the logarithm: half of them multiples of 64, the others as they fall."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if rng.random() < 0.5 and v >= 64 else v


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "linear_backward", "qk", "rope"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    if op in ("linear", "linear_backward"):
        m, k, n = _log(rng, 1, 4096), _size(rng, 48, 14336), _size(rng, 48, 14336)
        if op == "linear_backward":
            m = max(m, 16)
        # no drawn case costs more than the largest listed one (fp32 runs at a fraction of the bf16 rate)
        while m * k * n > 4096 * 4096 * 14336 // (8 if dtype == "f32" else 1):
            m, k = max(1, m // 2), max(48, k // 2)
        act = rng.choice(ACTS)
        if op == "linear":
            return dict(op=op, m=m, k=k, n=n, dtype=dtype, act=act, bias=rng.random() < 0.5,
                        residual=rng.choice(["none", "none", dtype, "f32"]),
                        save=act != "none" and rng.random() < 0.5)
        # An fp32 weight gradient of bf16 operands goes with a layer that has no activation of its own.
        dw = "f32" if dtype == "f32" or (act == "none" and rng.random() < 0.5) else "bf16"
        return dict(op=op, m=m, k=k, n=n, dtype=dtype, act=act, bias=rng.random() < 0.5, dw=dw)
    dim = rng.choice([64, 72, 80, 96, 112, 128, 128, 192, 256])
    hk = rng.choice([1, 2, 4, 8, 16])
    hq = hk * rng.choice([1, 2, 4, 7])
    tokens = _log(rng, 1, 30000)
    while tokens * (hq + hk) * dim > 30011 * 32 * 128 // (2 if dtype == "f32" else 1):
        tokens = max(1, tokens // 2)
    rot = dim if rng.random() < 0.7 else dim // 4 * 2
    case = dict(op=op, tokens=tokens, hq=hq, hk=hk, dim=dim, dtype=dtype, rot=rot,
                interleaved=rng.random() < 0.4, backward=rng.random() < 0.5, far=_log(rng, 64, 1000000))
    if op == "rope":
        case["axes"] = rng.choice([2, 3])
    return case


def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _sections(case):
    """Pairs per axis: 16, 24 and 24 of 64 for three axes, halves for two."""
    pairs, axes = case["rot"] // 2, case.get("axes", 1)
    if axes == 1:
        return [pairs]
    if axes == 2:
        return [pairs // 2, pairs - pairs // 2]
    first = pairs // 4
    second = (pairs - first) // 2
    return [first, second, pairs - first - second]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = _randn(gen, (m, k), dt)
        s["w"] = _randn(gen, (n, k), dt, 1 / math.sqrt(k))
        s["b"] = _randn(gen, (n,), dt, 0.1) if case["bias"] else None
        s["r"] = _randn(gen, (m, n), DTYPES[case["residual"]]) if case["residual"] != "none" else None
    elif case["op"] == "linear_backward":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = _randn(gen, (m, k), dt)
        s["w"] = _randn(gen, (n, k), dt, 1 / math.sqrt(k))
        s["dy"] = _randn(gen, (m, n), dt, 0.1)
        # the pre-activation as the forward pass left it
        s["z"] = _randn(gen, (m, n), dt) if case["act"] != "none" else None
    else:
        t, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["dim"]
        qkv = _randn(gen, (t, (hq + 2 * hk) * d), dt)  # packed rows, q and k are views of them
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        pairs = case["rot"] // 2
        s["sections"] = _sections(case)
        if case["op"] == "qk":
            s["wq"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
            s["wk"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
            # sequences packed one after the other, each counting from its own offset
            start = torch.randint(0, case["far"], (t // 512 + 1,), generator=gen, device="cuda")
            at = torch.arange(t, device="cuda")
            s["pos"] = start[at // 512] + at % 512
            order = torch.arange(pairs, device="cuda", dtype=torch.float64)
            s["inv_freq"] = torch.pow(500000.0, -order / pairs)
        else:
            s["pos"] = torch.randint(0, case["far"], (case["axes"], t), generator=gen, device="cuda")
            order = torch.arange(pairs, device="cuda", dtype=torch.float64)
            s["inv_freq"] = torch.pow(10000.0, -order / pairs)
        if case["backward"]:
            s["dq"] = _randn(gen, (t, hq, d), dt, 0.1)
            s["dk"] = _randn(gen, (t, hk, d), dt, 0.1)
    return s


# ---- the plain forms -----------------------------------------------------------

SQRT2 = math.sqrt(2.0)
TANH_A = math.sqrt(2.0 / math.pi)
TANH_B = 0.044715


def _act(z, name):
    if name == "relu":
        return z * (z > 0)
    if name == "relu2":
        return z * z * (z > 0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / SQRT2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(TANH_A * (z + TANH_B * z * z * z)))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "relu2":
        return 2 * z * (z > 0)
    if name == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z / SQRT2)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(TANH_A * (z + TANH_B * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * TANH_A * (1 + 3 * TANH_B * z * z)
    return torch.ones_like(z)


def _angles(s):
    """cos and sin of every token's pairs, [tokens, 1, pairs] in fp32 from fp64 angles."""
    pos, f = s["pos"], s["inv_freq"]
    if pos.dim() == 1:
        a = pos.double()[:, None] * f
    else:
        axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=pos.device),
                                       torch.tensor(s["sections"], device=pos.device))
        a = pos.double()[axis].t() * f
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _split(x, s):
    """The two members of every rotated pair and the rest of the head."""
    rot = s["rot"]
    if s["interleaved"]:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _join(a, b, rest, s):
    pair = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([pair, rest], -1)


def _rotate(x, cos, sin, s):
    a, b, rest = _split(x, s)
    return _join(a * cos - b * sin, b * cos + a * sin, rest, s)


EPS = 1e-6


def _norm_backward(g, x, w):
    """Gradients of x * rsqrt(mean(x^2) + eps) * w to x and w."""
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    gw = g * w
    return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum((0, 1))


def run(s):
    if own:
        return _run_own(s)
    dt = DTYPES[s["dtype"]]
    if s["op"] == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        y = y.to(dt if s["r"] is None else s["r"].dtype)
        return (y, z.to(dt)) if s["save"] else y
    if s["op"] == "linear_backward":
        g = s["dy"].float()
        if s["z"] is not None:
            g = g * _act_slope(s["z"].float(), s["act"])
        dx = (g @ s["w"].float()).to(dt)
        dw = (g.t() @ s["x"].float()).to(DTYPES[s["dw"]])
        return (dx, dw, g.sum(0).to(dt)) if s["bias"] else (dx, dw)
    cos, sin = _angles(s)
    if s["op"] == "rope":
        if s["backward"]:
            return [_rotate(g.float(), cos, -sin, s).to(dt) for g in (s["dq"], s["dk"])]
        return [_rotate(x.float(), cos, sin, s).to(dt) for x in (s["q"], s["k"])]
    both = ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk")))
    if not s["backward"]:
        out = []
        for x, w, _ in both:
            x = x.float()
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
            out.append(_rotate(x, cos, sin, s).to(dt))
        return out
    out = []
    for x, w, g in both:
        dx, dw = _norm_backward(_rotate(g.float(), cos, -sin, s), x.float(), w.float())
        out += [dx.to(dt), dw.to(dt)]
    return out


def _run_own(s):
    import newton_schulz_ns5_amd as ns
    act = None if s.get("act", "none") == "none" else s["act"]
    if s["op"] == "linear":
        return ns.linear(s["x"], s["w"], s["b"], s["r"], activation=act, return_preact=s["save"])
    if s["op"] == "linear_backward":
        dx, dw, db = ns.linear_backward(s["dy"], s["x"], s["w"], activation=act, preact=s["z"],
                                        need_dbias=s["bias"], dw_dtype=DTYPES[s["dw"]])
        return (dx, dw, db) if s["bias"] else (dx, dw)
    how = dict(interleaved=s["interleaved"])
    if s["op"] == "rope":
        how["sections"] = s["sections"]
        if s["backward"]:
            return list(ns.rope_backward(s["dq"], s["dk"], s["pos"], s["inv_freq"], **how))
        return list(ns.rope(s["q"], s["k"], s["pos"], s["inv_freq"], **how))
    if not s["backward"]:
        return list(ns.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_weight=s["wq"], k_weight=s["wk"],
                                    eps=EPS, **how))
    dq, dk, dwq, dwk = ns.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["inv_freq"],
                                                q_weight=s["wq"], k_weight=s["wk"], eps=EPS, **how)
    return [dq, dwq, dk, dwk]


# ---- what a pass cannot do without -----------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("linear", "linear_backward"):
        m, k, n = case["m"], case["k"], case["n"]
        if case["op"] == "linear":
            r = {"none": 0, "bf16": 2, "f32": 4}[case["residual"]]
            out = r if r else e
            return {"bytes": e * (m * k + n * k + (n if case["bias"] else 0) + (m * n if case["save"] else 0))
                    + (r + out) * m * n, "flops": 2 * m * k * n}
        z = e * m * n if case["act"] != "none" else 0
        return {"bytes": e * (m * n + m * k + n * k) + z + e * m * k + (4 if case["dw"] == "f32" else 2) * n * k
                + (e * n if case["bias"] else 0), "flops": 4 * m * k * n}
    rows = case["tokens"] * (case["hq"] + case["hk"])
    size = rows * case["dim"] * e
    pos = 8 * case["tokens"] * case.get("axes", 1)
    if case["op"] == "rope":
        return {"bytes": 2 * size + pos, "flops": 3 * rows * case["rot"]}
    if case["backward"]:
        return {"bytes": 3 * size + pos + 4 * e * case["dim"], "flops": rows * (3 * case["rot"] + 11 * case["dim"])}
    return {"bytes": 2 * size + pos + 2 * e * case["dim"], "flops": rows * (3 * case["rot"] + 4 * case["dim"])}


# ---- the definitions in 64 bits ----------------------------------------------------

def _exact_act(z, name):
    """The activation and its derivative."""
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    if name == "relu":
        return torch.maximum(z, zero), torch.where(z > 0, one, zero)
    if name == "relu2":
        p = torch.maximum(z, zero)
        return p * p, 2 * p
    if name == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg + z * sg * (1 - sg)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / 2.0 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2) / (2 * math.pi) ** 0.5
    if name == "gelu_tanh":
        # 1/2 (1 + tanh(u)) is the logistic function of 2 u
        c = (2 / math.pi) ** 0.5
        u = 2 * c * (z + 0.044715 * z ** 3)
        sg = torch.sigmoid(u)
        return z * sg, sg + z * sg * (1 - sg) * 2 * c * (1 + 3 * 0.044715 * z.square())
    return z, one


def _exact_rotation(pos, f, sections, rot, dim, interleaved):
    """Every token's rotation as complex factors and the place of every pair's members in the head."""
    pos = pos if pos.dim() == 2 else pos[None]
    cols, at = [], 0
    for axis, count in enumerate(sections):
        cols.append(pos[axis].double()[:, None] * f[None, at:at + count])
        at += count
    theta = torch.cat(cols, 1)
    p = torch.arange(rot // 2, device=pos.device)
    first, second = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
    return torch.polar(torch.ones_like(theta), theta)[:, None], first, second


def _exact_turn(x, turn, first, second):
    y = x.clone()
    c = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = c.real, c.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        z = torch.mm(s["x"].double(), s["w"].double().t())
        if s["b"] is not None:
            z += s["b"].double()
        y = _exact_act(z, case["act"])[0]
        if s["r"] is not None:
            y = y + s["r"].double()
        return (y, z) if case["save"] else y
    if case["op"] == "linear_backward":
        dz = s["dy"].double()
        if s["z"] is not None:
            dz = dz * _exact_act(s["z"].double(), case["act"])[1]
        dx, dw = torch.mm(dz, s["w"].double()), torch.mm(dz.t(), s["x"].double())
        return (dx, dw, dz.sum(0)) if case["bias"] else (dx, dw)
    turn, first, second = _exact_rotation(s["pos"], s["inv_freq"], s["sections"], case["rot"], case["dim"],
                                          case["interleaved"])
    if case["op"] == "rope":
        if case["backward"]:
            return [_exact_turn(g.double(), turn.conj(), first, second) for g in (s["dq"], s["dk"])]
        return [_exact_turn(x.double(), turn, first, second) for x in (s["q"], s["k"])]
    out = []
    for x, w, g in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x, w = x.double(), w.double()
        rms = (x.square().sum(-1, keepdim=True) / case["dim"] + EPS).sqrt()
        if not case["backward"]:
            out.append(_exact_turn(x / rms * w, turn, first, second))
            continue
        u = _exact_turn(g.double(), turn.conj(), first, second)
        dx = u * w / rms - x * (u * w * x).sum(-1, keepdim=True) / (case["dim"] * rms ** 3)
        out += [dx, (u * x / rms).sum((0, 1))]
    return out
