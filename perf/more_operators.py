"""Cases of what stands around a layer's products in a pass: the embedding
lookup with its gradient, the norms before and after a block with its gate and
its residual, and the norm over all gradients with their clipping.

`run` computes each in its plain form (elementary torch operations in fp32,
long sums in fp64, one rounding at the end) or, with `own` set, through this
package's entry points.  `exact` gives the same results in fp64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6       # of the norms
CLIP_EPS = 1e-6  # added to the gradient norm

# The matrices of one layer: q, k, v, o, gate, up and down of 4096 wide tokens with 32 query and 8 key heads
# of 128 and an MLP of 14336, and its two norms.
LAYER = "4096x4096 1024x4096 1024x4096 4096x4096 14336x4096 14336x4096 4096x14336 4096 4096"


def listed():
    return [
        # One token each of 16 sequences that decode together.
        dict(name="embedding decode", op="embedding", tokens=16, rows=131072, dim=4096, dtype="bf16", out="bf16",
             scale=1.0, shard=False),
        # A training batch of 8192 tokens into an fp32 residual stream, scaled by the root of the width.
        dict(name="embedding batch", op="embedding", tokens=8192, rows=131072, dim=4096, dtype="bf16", out="f32",
             scale=64.0, shard=False),
        # The gradient of such a batch over the whole vocabulary, in the weight's type.
        dict(name="embedding gradient batch", op="embedding_backward", tokens=8192, rows=131072, dim=4096,
             dtype="bf16", out="bf16", scale=1.0, shard=False),
        # The fp32 gradient of a long batch over one shard of a vocabulary (a quarter of the tokens are the shard's),
        # odd sizes, frequent tokens occurring thousands of times.
        dict(name="embedding gradient shard", op="embedding_backward", tokens=65537, rows=32003, dim=1001,
             dtype="f32", out="f32", scale=32.0, shard=True),
        # 16 decoding sequences between two blocks: norm of the block's output, onto the residual, next block's norm.
        dict(name="norms decode", op="norms", rows=16, cols=4096, seqs=1, dtype="bf16", stream="bf16", post=True,
             gate="none", pre=True, backward=False),
        # A training batch of 8192 tokens between two blocks, with a learned gate per column.
        dict(name="norms train", op="norms", rows=8192, cols=4096, seqs=1, dtype="bf16", stream="bf16", post=True,
             gate="cols", pre=True, backward=False),
        # Its gradients: block, residual, both norm weights and the gate.
        dict(name="norms train backward", op="norms", rows=8192, cols=4096, seqs=1, dtype="bf16", stream="bf16",
             post=True, gate="cols", pre=True, backward=True),
        # Gradients on an fp32 residual stream, five sequences of 1021 tokens each gated by its own row, odd width.
        dict(name="norms gated sequences", op="norms", rows=5105, cols=2050, seqs=5, dtype="bf16", stream="f32",
             post=False, gate="seqs", pre=True, backward=True),
        # The norm over the small parameters of a model (norm weights, biases): many tiny tensors.
        dict(name="gradient norm small", op="grad_norm", shapes=" ".join(["4096", "128", "1025", "33x17"] * 12), mix="f32"),
        # The norm over eight layers' gradients.
        dict(name="gradient norm 8 layers", op="grad_norm", shapes=" ".join([LAYER] * 8), mix="bf16"),
        # Clipping a small model's gradients of both types, odd sizes among them.
        dict(name="clip small model", op="clip", shapes=" ".join(["501x257", "768x768", "2049", "96x3x3x3"] * 6), mix="both"),
        # Clipping one layer's gradients.
        dict(name="clip layer", op="clip", shapes=LAYER, mix="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size spread over the logarithm: half of them multiples of 64, the others as they fall."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if rng.random() < 0.5 and v >= 64 else v


def draw(rng):
    op = rng.choice(["embedding", "embedding_backward", "embedding_backward", "norms", "norms", "norms", "grad_norm",
                     "clip", "clip"])
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    other = dtype if rng.random() < 0.6 else "f32"
    if op in ("embedding", "embedding_backward"):
        tokens, rows, dim = _log(rng, 1, 131072), _log(rng, 100, 262144), _size(rng, 16, 8192)
        while tokens * dim > 8192 * 4096:
            tokens = max(1, tokens // 2)
        while rows * dim > 131072 * 4096 // (2 if other == "f32" else 1):
            rows //= 2
        return dict(op=op, tokens=tokens, rows=rows, dim=dim, dtype=dtype, out=other,
                    scale=rng.choice([1.0, 1.0, math.sqrt(dim)]), shard=rng.random() < 0.3)
    if op == "norms":
        cols, seqs = _size(rng, 16, 16384), rng.choice([1, 1, 3, 8])
        rows = _log(rng, 1, 65536)
        while rows * cols > 8192 * 4096 // (2 if other == "f32" else 1):
            rows = max(1, rows // 2)
        rows = max(1, rows // seqs) * seqs
        gate = rng.choice(["none", "none", "cols", "seqs", "rows"])
        post, pre = rng.random() < 0.5, rng.random() < 0.85
        return dict(op=op, rows=rows, cols=cols, seqs=seqs, dtype=dtype, stream=other, post=post, gate=gate,
                    pre=pre, backward=rng.random() < 0.5)
    shapes, total, most = [], 0, _log(rng, 1000, 200_000_000)
    for _ in range(rng.randint(1, 60)):
        shape = (_size(rng, 16, 14336),) if rng.random() < 0.4 else (_size(rng, 16, 14336), _size(rng, 16, 8192))
        if total + math.prod(shape) <= most or not shapes:
            shapes.append("x".join(map(str, shape)))
            total += math.prod(shape)
    return dict(op=op, shapes=" ".join(shapes), mix=rng.choice(["bf16", "f32", "both"]))


def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _ids(gen, case):
    """Token numbers whose frequency falls with their rank (Zipf's law), as texts have; of a shard: its quarter of
    a vocabulary four times as large, the second one, every fourth token being the shard's at the same law."""
    u = torch.rand(case["tokens"], generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(case["rows"] + 1)) - 1).long().clamp_(0, case["rows"] - 1)
    if case["shard"]:
        quarter = torch.randint(0, 4, (case["tokens"],), generator=gen, device="cuda")
        ids = ids + quarter * case["rows"]
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]] if "dtype" in case else None
    s = dict(case)
    if case["op"] in ("embedding", "embedding_backward"):
        s["ids"] = _ids(gen, case)
        s["first"] = case["rows"] if case["shard"] else 0
        if case["op"] == "embedding":
            s["w"] = _randn(gen, (case["rows"], case["dim"]), dt, 0.02)
        else:
            s["dy"] = _randn(gen, (case["tokens"], case["dim"]), dt, 0.1)
    elif case["op"] == "norms":
        r, c, st = case["rows"], case["cols"], DTYPES[case["stream"]]
        shape = (case["seqs"], r // case["seqs"], c)
        s["block"] = _randn(gen, shape, dt)
        s["w"] = (1 + 0.1 * torch.randn(c, generator=gen, device="cuda")).to(dt) if case["pre"] else None
        s["post_w"] = (1 + 0.1 * torch.randn(c, generator=gen, device="cuda")).to(dt) if case["post"] else None
        lead = {"none": None, "cols": (), "seqs": (case["seqs"], 1), "rows": shape[:2]}[case["gate"]]
        s["g"] = _randn(gen, lead + (c,), dt, 0.5) if lead is not None else None
        if case["backward"]:
            # the stream as the forward pass left it, the gradients of both results
            s["stream_out"] = _randn(gen, shape, st, 2.0) if case["pre"] else None
            s["dy"] = _randn(gen, shape, dt, 0.1) if case["pre"] else None
            s["dstream"] = _randn(gen, shape, st, 0.1)
        else:
            s["x"] = _randn(gen, shape, st, 2.0)
    else:
        shapes = [tuple(map(int, t.split("x"))) for t in case["shapes"].split()]
        kinds = [DTYPES["f32" if case["mix"] == "f32" or (case["mix"] == "both" and len(t) < 2) else "bf16"] for t in shapes]
        s["grads"] = [_randn(gen, t, k, 0.01) for t, k in zip(shapes, kinds)]
        if case["op"] == "clip":
            # clipped to 0.37 of it; into buffers of the optimizer's, so that every pass has the same gradients
            s["max_norm"] = 0.0037 * math.sqrt(sum(map(math.prod, shapes)))
            s["out"] = [torch.empty_like(g) for g in s["grads"]]
    return s


# What multiplies the residual and the block's output: as scaled residual streams have them.
RESIDUAL_SCALE, BLOCK_SCALE = 1.0, 0.75


# ---- the plain forms -----------------------------------------------------------

def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _norm_backward(g, x, w):
    """Gradients of x * rsqrt(mean(x^2) + eps) * w to x and w."""
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    gw = g * w
    return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum((0, 1), dtype=torch.float64)


def _gate_sum(p, s):
    """The gate's gradient from the one that a gate for every row would have."""
    if s["gate"] == "cols":
        return p.sum((0, 1), dtype=torch.float64)
    return p.sum(1, keepdim=True, dtype=torch.float64) if s["gate"] == "seqs" else p


def _shard(s):
    """Every token's row in the shard, and whether it has one."""
    at = s["ids"] - s["first"]
    inside = (at >= 0) & (at < s["rows"])
    return torch.where(inside, at, 0), inside[:, None]


def _global_norm(grads):
    return torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt()


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "embedding":
        at, inside = _shard(s)
        return (s["w"][at].float() * s["scale"] * inside).to(DTYPES[s["out"]])
    if s["op"] == "embedding_backward":
        at, inside = _shard(s)
        dw = torch.zeros(s["rows"], s["dim"], device=at.device)
        return dw.index_add_(0, at, s["dy"].float() * inside).mul_(s["scale"]).to(DTYPES[s["out"]])
    if s["op"] == "grad_norm":
        return _global_norm(s["grads"]).float()
    if s["op"] == "clip":
        norm = _global_norm(s["grads"])
        f = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0).float()
        return [norm.float()] + [o.copy_(g.float() * f) for g, o in zip(s["grads"], s["out"])]
    dt, st = DTYPES[s["dtype"]], DTYPES[s["stream"]]
    b = s["block"].float()
    if not s["backward"]:
        u = _norm(b, s["post_w"].float()) if s["post"] else b
        if s["g"] is not None:
            u = u * s["g"].float()
        x = RESIDUAL_SCALE * s["x"].float() + BLOCK_SCALE * u
        return [x.to(st), _norm(x, s["w"].float()).to(dt)] if s["pre"] else [x.to(st)]
    d, out = s["dstream"].float(), {}
    if s["pre"]:
        dn, dw = _norm_backward(s["dy"].float(), s["stream_out"].float(), s["w"].float())
        d = d + dn
        out["dweight"] = dw.to(dt)
    out["dresidual"] = (RESIDUAL_SCALE * d).to(st)
    du = BLOCK_SCALE * d
    if s["g"] is not None:
        u = _norm(b, s["post_w"].float()) if s["post"] else b
        out["dgate"] = _gate_sum(du * u, s).to(dt)
        du = du * s["g"].float()
    if s["post"]:
        du, dw = _norm_backward(du, b, s["post_w"].float())
        out["dpost_weight"] = dw.to(dt)
    out["dblock"] = du.to(dt)
    return out


def _run_own(s):
    import newton_schulz_ns5_amd as ns
    if s["op"] == "embedding":
        return ns.embedding(s["ids"], s["w"], scale=s["scale"], first=s["first"], dtype=DTYPES[s["out"]])
    if s["op"] == "embedding_backward":
        return ns.embedding_backward(s["dy"], s["ids"], s["rows"], scale=s["scale"], first=s["first"],
                                     dw_dtype=DTYPES[s["out"]])
    if s["op"] == "grad_norm":
        return ns.grad_norm(s["grads"])
    if s["op"] == "clip":
        return [ns.clip_grad_norm(s["grads"], s["max_norm"], eps=CLIP_EPS, out=s["out"])] + s["out"]
    how = dict(weight=s["w"], post_weight=s["post_w"], gate=s["g"], norm=s["pre"], post_norm=s["post"],
               scale=BLOCK_SCALE, residual_scale=RESIDUAL_SCALE, eps=EPS)
    if not s["backward"]:
        stream, y = ns.residual_norm(s["block"], s["x"], **how)
        return [stream, y] if s["pre"] else [stream]
    got = ns.residual_norm_backward(s["dy"], s["dstream"], s["stream_out"], s["block"], **how)
    names = ("dblock", "dresidual", "dweight", "dpost_weight", "dgate")
    return {n: t for n, t in zip(names, got) if t is not None}


# ---- what a pass cannot do without -----------------------------------------------

def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] in ("embedding", "embedding_backward"):
        t, d, e, o = case["tokens"], case["dim"], size[case["dtype"]], size[case["out"]]
        mine = t / 4 if case["shard"] else t  # tokens that have a row
        if case["op"] == "embedding":
            return {"bytes": 8 * t + min(mine, case["rows"]) * d * e + t * d * o, "flops": mine * d}
        return {"bytes": 8 * t + mine * d * e + case["rows"] * d * o, "flops": 2 * mine * d}
    if case["op"] in ("grad_norm", "clip"):
        shapes = [tuple(map(int, t.split("x"))) for t in case["shapes"].split()]
        each = [math.prod(t) * (4 if case["mix"] == "f32" or (case["mix"] == "both" and len(t) < 2) else 2) for t in shapes]
        n = sum(map(math.prod, shapes))
        return {"bytes": sum(each) * (2 if case["op"] == "clip" else 1) + 4, "flops": n * (3 if case["op"] == "clip" else 2)}
    n, e, r = case["rows"] * case["cols"], size[case["dtype"]], size[case["stream"]]
    gate = {"none": 0, "cols": case["cols"], "seqs": case["seqs"] * case["cols"], "rows": n}[case["gate"]] * e
    vectors = (case["post"] + case["pre"]) * case["cols"] * e + gate
    if not case["backward"]:
        return {"bytes": n * (e + 2 * r + (e if case["pre"] else 0)) + vectors,
                "flops": n * (3 + 4 * case["post"] + 4 * case["pre"])}
    needs_block = case["post"] or case["gate"] != "none"
    return {"bytes": n * ((e if needs_block else 0) + (e + r if case["pre"] else 0) + r + e + r) + 2 * vectors,
            "flops": n * (3 + 11 * case["post"] + 11 * case["pre"])}


# ---- the definitions in 64 bits ----------------------------------------------------

def _exact_norm(x, w):
    return x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embedding":
        y = torch.zeros(case["tokens"], case["dim"], device="cuda", dtype=torch.float64)
        mine = ((s["ids"] >= s["first"]) & (s["ids"] < s["first"] + case["rows"])).nonzero()[:, 0]
        y[mine] = case["scale"] * s["w"].index_select(0, s["ids"][mine] - s["first"]).double()
        return y
    if case["op"] == "embedding_backward":
        dw = torch.zeros(case["rows"], case["dim"], device="cuda", dtype=torch.float64)
        mine = ((s["ids"] >= s["first"]) & (s["ids"] < s["first"] + case["rows"])).nonzero()[:, 0]
        return dw.index_put_((s["ids"][mine] - s["first"],), case["scale"] * s["dy"][mine].double(), accumulate=True)
    if case["op"] in ("grad_norm", "clip"):
        total = 0.0
        for g in s["grads"]:
            total += float(torch.linalg.vector_norm(g.double())) ** 2
        norm = torch.tensor(math.sqrt(total), dtype=torch.float64)
        if case["op"] == "grad_norm":
            return norm
        f = min(1.0, s["max_norm"] / (math.sqrt(total) + CLIP_EPS))
        return [norm] + [g.double() * f for g in s["grads"]]
    # the backward pass by differentiating the forward definition
    b = s["block"].double().requires_grad_(case["backward"])
    vectors = {n: (s[n].double().requires_grad_(case["backward"]) if s[n] is not None else None) for n in ("w", "post_w", "g")}
    u = _exact_norm(b, vectors["post_w"]) if case["post"] else b
    u = u * vectors["g"] if vectors["g"] is not None else u
    if not case["backward"]:
        x = RESIDUAL_SCALE * s["x"].double() + BLOCK_SCALE * u
        return [x, _exact_norm(x, vectors["w"])] if case["pre"] else [x]
    out, d = {}, s["dstream"].double()
    if case["pre"]:
        x = s["stream_out"].double().requires_grad_()
        dx, out["dweight"] = torch.autograd.grad(_exact_norm(x, vectors["w"]), (x, vectors["w"]), s["dy"].double())
        d = d + dx
    out["dresidual"] = RESIDUAL_SCALE * d
    names = [n for n in ("g", "post_w") if vectors[n] is not None]
    got = torch.autograd.grad(u, [b] + [vectors[n] for n in names], BLOCK_SCALE * d) if names else [BLOCK_SCALE * d]
    out["dblock"] = got[0]
    for n, t in zip(names, got[1:]):
        out[{"g": "dgate", "post_w": "dpost_weight"}[n]] = t
    return out
