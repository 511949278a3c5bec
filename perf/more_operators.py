"""What is measured of the feed-forward half of a decoder layer and of the end of a training step:
the cases, their inputs, the plain forms, and the definitions in 64 bits.

Operators (``case["op"]``):

norm, norm_grad
    Layer norm of rows: y = (x - mean) / sqrt(var + eps) * w + b; its gradient gives the inputs', the
    weight's and the bias's.
ffn, ffn_train
    Gated feed-forward block: H = act(X Wg) * (X Wu); the training step returns H and the gradients of
    X, Wg and Wu for a given gradient of H.
clip
    The global 2-norm of many gradient tensors, and the tensors times min(1, max_norm / (norm + 1e-6)).
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
CLIP_EPS = 1e-6
MOST_FLOPS = 12 * 4096 * 4096 * 14336      # of a gated block's case
MOST_CLIP = 218 << 20                      # elements of a clipping case


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of four sequences: latency
        dict(name="norm-token", op="norm", rows=4, d=4096, bias=True, dtype="bf16"),
        # a ragged batch of rows in a wider buffer
        dict(name="norm-ragged", op="norm", rows=5003, d=3584, bias=False, dtype="fp16"),
        # a training batch's forward
        dict(name="norm-batch", op="norm", rows=16384, d=4096, bias=True, dtype="bf16"),
        # the gradient in 32 bits at an odd width
        dict(name="norm-grad-odd", op="norm_grad", rows=3001, d=1999, bias=True, dtype="fp32"),
        # the training batch's gradient
        dict(name="norm-grad", op="norm_grad", rows=16384, d=4096, bias=True, dtype="bf16"),
        # one decoding step of eight sequences: the weights' bytes count
        dict(name="ffn-token", op="ffn", rows=8, d=4096, d_ff=14336, act="silu", dtype="bf16"),
        # a short prompt through one shard of the weights
        dict(name="ffn-few", op="ffn", rows=203, d=3584, d_ff=2368, act="gelu_tanh", dtype="fp16"),
        # long prompts
        dict(name="ffn-prompt", op="ffn", rows=8192, d=4096, d_ff=14336, act="silu", dtype="bf16"),
        # a training step on an odd number of tokens through one shard of the weights
        dict(name="ffn-train-ragged", op="ffn_train", rows=1003, d=3584, d_ff=2368, act="gelu_tanh", dtype="fp16"),
        # a training step with whole weights
        dict(name="ffn-train", op="ffn_train", rows=4096, d=4096, d_ff=14336, act="silu", dtype="bf16"),
        # the norms' weights and small projections alone: latency
        dict(name="clip-few", op="clip", tensors=24, total=100003, mix="fp32", max_norm=1.0, shape=1),
        # a decoder layer's gradients in 32 bits (attention 4096 x 6144 and 4096 x 4096, three of 4096 x 14336, norms)
        dict(name="clip-layer", op="clip", tensors=9, total=0, mix="fp32", max_norm=1.0, shape=0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_grad", "ffn", "ffn", "ffn_train", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("norm", "norm_grad"):
        d = rng.choice([rng.randrange(16, 512), log(64, 8192), log(64, 8192), 8 * log(8, 1024), 8 * log(8, 2048)])
        dtype = rng.choice([dtype, dtype, "fp32"])
        most = 16384 * 4096 * 2 // (d * (4 if dtype == "fp32" else 2))
        return dict(op=op, rows=min(log(1, most), 1 << 20), d=d, bias=rng.random() < 0.6, dtype=dtype)
    if op == "clip":
        return dict(op=op, tensors=log(1, 400), total=log(1, MOST_CLIP // 4),
                    mix=rng.choice(["fp32", "bf16", "fp16", "all"]), max_norm=rng.choice([0.3, 1.0, 1e6]),
                    shape=rng.randrange(1, 1 << 20))
    d, d_ff = 8 * log(8, 1024), 8 * log(8, 2048)
    most = MOST_FLOPS // ((4 if op == "ffn" else 12) * d * d_ff)
    return dict(op=op, rows=log(1, max(min(most, 16384), 1)), d=d, d_ff=d_ff,
                act=rng.choice(["silu", "silu", "gelu_tanh", "gelu"]), dtype=dtype)


def _tensors(case):
    """(elements, type) of each tensor of a clipping case."""
    if case["shape"] == 0:
        sizes = [4096 * 6144, 4096 * 4096] + [4096 * 14336] * 3 + [4096, 4096, 128, 128]
        return [(n, case["mix"]) for n in sizes]
    rng = random.Random(case["shape"])
    # a few large ones and many small ones, as a model has
    share = [math.exp(rng.uniform(0, 7)) for _ in range(case["tensors"])]
    scale = case["total"] / sum(share)
    kinds = ["fp32", "bf16", "fp16"] if case["mix"] == "all" else [case["mix"]]
    return [(int(s * scale), rng.choice(kinds)) for s in share]


def work(case):
    c = case
    if c["op"] == "clip":
        t = _tensors(c)
        return {"bytes": sum(n * (4 if k == "fp32" else 2) * 2 for n, k in t) + 4, "flops": 3 * sum(n for n, _ in t)}
    size = 4 if c["dtype"] == "fp32" else 2
    n = c["rows"] * c["d"]
    if c["op"] == "norm":
        return {"bytes": n * 2 * size + c["d"] * size * (2 if c["bias"] else 1), "flops": 8 * n}
    if c["op"] == "norm_grad":
        return {"bytes": n * 3 * size + c["d"] * (size + (8 if c["bias"] else 4)), "flops": 16 * n}
    w, h = c["d"] * c["d_ff"], c["rows"] * c["d_ff"]
    if c["op"] == "ffn":
        return {"bytes": (n + h + 2 * w) * size, "flops": 4 * c["rows"] * w}
    # X, dX, H, dH, the weights and their gradients once each
    return {"bytes": (2 * n + 2 * h + 4 * w) * size, "flops": 12 * c["rows"] * w}


# ---------------------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    if c["op"] == "clip":
        # gradients of different layers differ in size
        return {"grads": [(normal(n) * 0.01 * 4.0 ** (i % 3 - 1)).to(TYPES[k]) for i, (n, k) in enumerate(_tensors(c))]}
    dt, rows, d = TYPES[c["dtype"]], c["rows"], c["d"]
    x = {}
    if c["op"] in ("norm", "norm_grad"):
        # residual rows: a mean, and a scale of their own; the rows lie in a wider buffer
        wide = torch.empty(rows, d + (16 if c["dtype"] == "fp16" else 0), dtype=dt, device="cuda")
        x["x"] = wide[:, :d]
        x["x"].copy_((normal(rows, d) + 0.3) * (0.5 + torch.rand(rows, 1, generator=g, device="cuda")))
        x["w"] = (1 + 0.2 * normal(d)).to(dt)
        x["b"] = (0.2 * normal(d)).to(dt) if c["bias"] else None
        if c["op"] == "norm_grad":
            x["dy"] = normal(rows, d).to(dt)
        return x
    f = c["d_ff"]
    x["x"] = normal(rows, d).to(dt)
    x["wg"], x["wu"] = ((normal(d, f) * d ** -0.5).to(dt) for _ in range(2))
    if c["op"] == "ffn_train":
        x["dh"] = normal(rows, f).to(dt)
    return x


def prepare(case, seed):
    c, x = case, _inputs(case, seed)
    s = {"case": c, **x}
    new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")
    if c["op"] == "clip":
        s["out"] = [torch.empty_like(t) for t in x["grads"]]
        s["norm"] = new(1, dtype=torch.float32)
        if own:
            from chunk_scheduled_communication_gb300 import clip
            s["plan"] = clip.ClipPlan()
        return s
    dt, rows, d = TYPES[c["dtype"]], c["rows"], c["d"]
    if c["op"] in ("norm", "norm_grad"):
        s["out"] = new(rows, d, dtype=dt)
        if c["op"] == "norm_grad":
            s["dw"] = new(d, dtype=torch.float32)
            s["db"] = new(d, dtype=torch.float32) if c["bias"] else None
        if own:
            from chunk_scheduled_communication_gb300 import norm
            s["plan"] = norm.NormPlan(d=d, dtype=c["dtype"])
        return s
    f = c["d_ff"]
    s["h"] = new(rows, f, dtype=dt)
    if c["op"] == "ffn_train":
        s["g"], s["u"], s["dx"] = new(rows, f, dtype=dt), new(rows, f, dtype=dt), new(rows, d, dtype=dt)
        s["dwg"], s["dwu"] = new(d, f, dtype=dt), new(d, f, dtype=dt)
    if own:
        from chunk_scheduled_communication_gb300 import ffn
        s["plan"] = ffn.FfnPlan(d=d, d_ff=f, act=c["act"], dtype=c["dtype"])
    return s


# ---------------------------------------------------------------------------------------- plain forms
def _act(kind, g):
    """act(g) and its derivative."""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _plain_norm(s):
    c, x, w = s["case"], s["x"].float(), s["w"].float()
    m = x.mean(-1, keepdim=True)
    x = x - m
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    x = x * r
    if c["op"] == "norm":
        y = x * w
        return (y if s["b"] is None else y + s["b"].float()).to(s["x"].dtype)
    dy = s["dy"].float()
    g = dy * w
    dx = r * (g - g.mean(-1, keepdim=True) - x * (g * x).mean(-1, keepdim=True))
    out = (dx.to(s["x"].dtype), (dy * x).sum(0))
    return out if s["b"] is None else out + (dy.sum(0),)


def _plain_ffn(s):
    c, dt = s["case"], s["x"].dtype
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg, x @ wu
    a, da = _act(c["act"], g)
    h = (a * u).to(dt)
    if c["op"] == "ffn":
        return h
    dh = s["dh"].float()
    dg, du = dh * u * da, dh * a
    return h, (dg @ wg.T + du @ wu.T).to(dt), (x.T @ dg).to(dt), (x.T @ du).to(dt)


def _plain_clip(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in s["grads"]:
        total = total + t.float().square().sum(dtype=torch.float64)
    norm = total.sqrt()
    k = (s["case"]["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
    return [norm.float().view(1)] + [(t.float() * k).to(t.dtype) for t in s["grads"]]


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_clip(s) if c["op"] == "clip" else _plain_norm(s) if c["op"] in ("norm", "norm_grad") else _plain_ffn(s)
    plan = s["plan"]
    if c["op"] == "clip":
        plan.clip(s["grads"], c["max_norm"], s["norm"], out=s["out"], eps=CLIP_EPS)
        return [s["norm"]] + s["out"]
    if c["op"] == "norm":
        plan.forward(s["x"], s["out"], s["w"], s["b"], eps=EPS)
        return s["out"]
    if c["op"] == "norm_grad":
        plan.backward(s["x"], s["dy"], s["out"], s["w"], s["dw"], s["db"], eps=EPS)
        return (s["out"], s["dw"]) if s["b"] is None else (s["out"], s["dw"], s["db"])
    if c["op"] == "ffn":
        plan.forward(s["x"], s["wg"], s["wu"], s["h"])
        return s["h"]
    plan.forward(s["x"], s["wg"], s["wu"], s["h"], G=s["g"], U=s["u"])
    # in place: the gradients of the projections take the projections' place
    plan.backward(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"], s["g"], s["u"], s["dx"], s["dwg"], s["dwu"])
    return s["h"], s["dx"], s["dwg"], s["dwu"]


# ---------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    c, x = case, _inputs(case, seed)
    if c["op"] == "clip":
        g = [t.double() for t in x["grads"]]
        norm = math.sqrt(sum(float(torch.dot(t, t)) for t in g))
        k = min(1.0, c["max_norm"] / (norm + CLIP_EPS))
        return [torch.tensor([norm], dtype=torch.float64, device="cuda")] + [t * k for t in g]
    want = c["op"] in ("norm_grad", "ffn_train")
    if c["op"] in ("norm", "norm_grad"):
        t, w = x["x"].double().requires_grad_(want), x["w"].double().requires_grad_(want)
        b = torch.zeros(c["d"], dtype=torch.float64, device="cuda") if x["b"] is None else x["b"].double()
        b.requires_grad_(want)
        var, mean = torch.var_mean(t, -1, unbiased=False, keepdim=True)
        y = (t - mean) / torch.sqrt(var + EPS) * w + b
        if not want:
            return y
        grads = torch.autograd.grad(y, [t, w, b], x["dy"].double())
        return grads[:2] if x["b"] is None else grads
    t, wg, wu = (x[k].double().requires_grad_(want) for k in ("x", "wg", "wu"))
    f = torch.nn.functional
    act = {"silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[c["act"]]
    h = act(t @ wg) * (t @ wu)
    if not want:
        return h
    return (h.detach(),) + torch.autograd.grad(h, [t, wg, wu], x["dh"].double())
