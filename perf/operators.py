"""What is measured of the operators in front of and behind a windowed attention: the cases, their
inputs, the plain forms, and the definitions in 64 bits.

Operators (``case["op"]``):

rope, rope_grad
    Rotary positions of the query and key heads: pairs (2i, 2i+1) ("interleaved") or (i, i + rot/2)
    ("half") of the first ``rot`` elements of a head turn by position * f_i; the rest passes through.
    f_i = base^(-2i/rot), scaled for long contexts ("none", "linear", "llama3", "yarn").
norm, norm_grad
    Root-mean-square norm of each query and key head with a weight per element, then the same
    rotation, in one pass; its gradient gives the inputs' and the weights'.
window, window_train
    Causal attention of ragged sequences in which query position p sees keys (p - W, p] and the first
    ``sinks`` keys; the training step returns the output and the gradients of Q, K and V.
decode
    One query token per sequence over a paged cache, same window and sinks.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 512     # query rows that the plain attention handles at once
EPS = 1e-6
BASE = 500000.0


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of eight sequences, part of the head rotated in adjacent pairs: latency
        dict(name="rope-token", op="rope", tokens=8, hq=32, hkv=8, d=128, rot=64, layout="interleaved",
             scaling="none", max_pos=8192, dtype="bf16"),
        # a long prompt beyond the trained context
        dict(name="rope-prompt", op="rope", tokens=32768, hq=32, hkv=8, d=128, rot=128, layout="half",
             scaling="yarn", max_pos=131072, dtype="bf16"),
        # the gradient in a training step with an odd number of tokens and grouped heads
        dict(name="rope-grad", op="rope_grad", tokens=5003, hq=28, hkv=4, d=128, rot=128, layout="half",
             scaling="llama3", max_pos=65536, dtype="fp16"),
        # one decoding step of four sequences: latency
        dict(name="norm-token", op="norm", tokens=4, hq=32, hkv=8, d=128, rot=128, layout="half",
             scaling="none", max_pos=32768, dtype="bf16"),
        # a training batch's forward
        dict(name="norm-batch", op="norm", tokens=16384, hq=32, hkv=8, d=128, rot=128, layout="half",
             scaling="none", max_pos=8192, dtype="bf16"),
        # the same batch's gradient
        dict(name="norm-grad", op="norm_grad", tokens=16384, hq=32, hkv=8, d=128, rot=128, layout="half",
             scaling="none", max_pos=8192, dtype="bf16"),
        # ragged prompts, one of them the continuation of a cached prefix, one longer than its keys; small heads
        dict(name="window-ragged", op="window", q_lens="1,129,700,2049,333,64", k_lens="1,129,700,2049,1500,40",
             hq=16, hkv=16, d=64, window=500, sinks=5, dtype="fp16"),
        # one long prompt
        dict(name="window-prompt", op="window", q_lens="16384", k_lens="16384", hq=32, hkv=8, d=128, window=4096,
             sinks=4, dtype="bf16"),
        # a packed batch of short documents, odd lengths, odd group of heads
        dict(name="train-ragged", op="window_train", q_lens="1024,517,63,1531", k_lens="1024,517,63,1531", hq=14,
             hkv=2, d=128, window=300, sinks=16, dtype="bf16"),
        # a training step on one long sequence
        dict(name="train-long", op="window_train", q_lens="16384", k_lens="16384", hq=32, hkv=8, d=128, window=2048,
             sinks=4, dtype="bf16"),
        # a decoding step of three sequences: latency
        dict(name="decode-few", op="decode", batch=3, max_len=5000, min_len=1, hq=32, hkv=8, d=128, window=1024,
             sinks=4, page=16, dtype="bf16"),
        # a full serving batch over long sequences
        dict(name="decode-batch", op="decode", batch=128, max_len=32768, min_len=6000, hq=32, hkv=8, d=128, window=4096,
             sinks=4, page=64, dtype="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "rope_grad", "norm", "norm_grad", "window", "window", "window_train", "window_train",
                     "decode", "decode"])
    hkv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("rope", "rope_grad", "norm", "norm_grad"):
        d = rng.choice([64, 128, 128, 256])
        hq = hkv * rng.choice([1, 2, 4, 7])
        most = 32 * 16384 * 128 // (max(hq, 8) * d)
        rot = rng.choice([d, d, d // 2])
        return dict(op=op, tokens=log(1, most), hq=hq, hkv=hkv, d=d, rot=rot,
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "llama3", "yarn"]), max_pos=log(40000, 1000000),
                    dtype=rng.choice([dtype, dtype, "fp32"]))
    d = rng.choice([64, 128, 128])
    hq = hkv * rng.choice([1, 2, 4, 4, 7]) if hkv < 8 else hkv * rng.choice([1, 2, 4])
    if op == "decode":
        batch = log(1, 128)
        lo = log(1, 4000)
        return dict(op=op, batch=batch, min_len=lo, max_len=lo + log(1, 16000), hq=hq, hkv=hkv, d=d,
                    window=log(64, 4096), sinks=rng.choice([0, 1, 4, 4, 13, 64]), page=rng.choice([16, 32, 64, 128]),
                    dtype=dtype)
    n = rng.choice([1, 1, 2, 3, 5])
    total = log(64, 16384)
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    q_lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    more = [rng.choice([0, 0, 0, log(1, 1000)]) if op == "window" else 0 for _ in range(n)]
    return dict(op=op, q_lens=",".join(map(str, q_lens)), k_lens=",".join(str(q + m) for q, m in zip(q_lens, more)),
                hq=hq, hkv=hkv, d=d, window=log(64, 2048), sinks=rng.choice([0, 1, 4, 4, 16, 50]), dtype=dtype)


def _lens(case, key):
    return [int(x) for x in str(case[key]).split(",")]


def _pairs(q_len, k_len, window, sinks):
    """How many (query, visible key) pairs a sequence has."""
    p = torch.arange(k_len - q_len, k_len, dtype=torch.int64)
    p = p[p >= 0]
    lo = (p - window + 1).clamp(min=0)
    return int((p + 1 - lo + torch.minimum(lo, torch.full_like(lo, sinks))).sum())


def work(case):
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    if "tokens" in c:
        heads = c["hq"] + c["hkv"]
        n = c["tokens"] * heads * c["d"]
        # forward and rope's gradient: each element read and written; the norm's gradient reads x and dy
        passes = 3 if c["op"] == "norm_grad" else 2
        flops = {"rope": 3, "rope_grad": 3, "norm": 7, "norm_grad": 14}[c["op"]]
        extra = {"norm": 2 * c["d"] * size, "norm_grad": 2 * c["d"] * (size + 4)}.get(c["op"], 0)
        return {"bytes": n * size * passes + c["tokens"] * 8 + extra, "flops": n * flops}
    if c["op"] == "decode":
        lens = _decode_lens(c, 0)
        seen = sum(_pairs(1, n, c["window"], c["sinks"]) for n in lens)
        io = 2 * c["batch"] * c["hq"] * c["d"] * size
        return {"bytes": 2 * seen * c["hkv"] * c["d"] * size + io, "flops": 4 * seen * c["hq"] * c["d"]}
    q, k = _lens(c, "q_lens"), _lens(c, "k_lens")
    pairs = sum(_pairs(a, b, c["window"], c["sinks"]) for a, b in zip(q, k))
    nq, nk = sum(q) * c["hq"] * c["d"], sum(k) * c["hkv"] * c["d"]
    if c["op"] == "window":
        return {"bytes": (2 * nq + 2 * nk) * size, "flops": 4 * pairs * c["hq"] * c["d"]}
    # two products forward, five backward; Q, dO, O, dQ and K, V, dK, dV once each
    return {"bytes": (4 * nq + 4 * nk) * size, "flops": 14 * pairs * c["hq"] * c["d"]}


# ---------------------------------------------------------------------------------------- inputs
def _scaling(case):
    return {"none": None,
            "linear": dict(kind="linear", factor=4.0),
            "llama3": dict(kind="llama3", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original_context=8192),
            "yarn": dict(kind="yarn", factor=4.0, original_context=32768, beta_fast=32.0, beta_slow=1.0)}[case["scaling"]]


def _frequencies(case):
    """f_i in radians per position (64 bits) and the factor on the rotated part."""
    rot, s = case["rot"], _scaling(case)
    f = torch.tensor(BASE, dtype=torch.float64) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if s is None:
        return f, 1.0
    if s["kind"] == "linear":
        return f / s["factor"], 1.0
    if s["kind"] == "llama3":
        wave = 2 * math.pi / f
        t = (s["original_context"] / wave - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])
        t = t.clamp(0, 1)
        return (1 - t) * f / s["factor"] + t * f, 1.0

    def index(turns):
        return rot * math.log(s["original_context"] / (turns * 2 * math.pi)) / (2 * math.log(BASE))

    low = max(math.floor(index(s["beta_fast"])), 0)
    high = min(math.ceil(index(s["beta_slow"])), rot - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f / s["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(s["factor"]) + 1.0


def _decode_lens(case, seed):
    """Lengths spread evenly over [min_len, max_len], the same for every seed."""
    b, lo, hi = case["batch"], case["min_len"], case["max_len"]
    return [lo + (hi - lo) * i // max(b - 1, 1) for i in range(b)]


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)
    dt = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    x = {}
    if "tokens" in c:
        t, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
        # queries, keys and values come out of one projection: rows of (hq + 2 hkv) heads
        qkv = normal(t, hq + 2 * hkv, d)
        x["q"], x["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        start = torch.randint(0, max(c["max_pos"] - t, 1), (1,), generator=g, device="cuda")
        # a decoding step has a position for each sequence, a batch runs of consecutive ones
        x["pos"] = (torch.randint(0, c["max_pos"], (t,), generator=g, device="cuda") if t <= 64 else
                    (start + torch.arange(t, device="cuda")) % c["max_pos"])
        if c["op"] in ("rope_grad", "norm_grad"):
            x["dq"], x["dk"] = normal(t, hq, d), normal(t, hkv, d)
        if c["op"] in ("norm", "norm_grad"):
            x["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
            x["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        return x
    if c["op"] == "decode":
        b, page = c["batch"], c["page"]
        lens = _decode_lens(c, seed)
        per = (max(lens) + page - 1) // page
        pages = sum((n + page - 1) // page for n in lens) + 8
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(b, per, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(lens):
            m = (n + page - 1) // page
            table[i, :m] = order[at:at + m]
            at += m
        x["q"] = normal(b, c["hq"], c["d"])
        x["k"], x["v"] = normal(pages, page, c["hkv"], c["d"]), normal(pages, page, c["hkv"], c["d"])
        x["table"], x["lens"] = table, torch.tensor(lens, dtype=torch.int32, device="cuda")
        return x
    nq, nk = sum(_lens(c, "q_lens")), sum(_lens(c, "k_lens"))
    x["q"], x["k"], x["v"] = normal(nq, c["hq"], c["d"]), normal(nk, c["hkv"], c["d"]), normal(nk, c["hkv"], c["d"])
    if c["op"] == "window_train":
        x["do"] = normal(nq, c["hq"], c["d"])
    return x


def prepare(case, seed):
    c, x = case, _inputs(case, seed)
    s = {"case": c, **x}
    new = torch.empty
    if "tokens" in c:
        if c["op"] in ("rope", "norm"):
            s["out"] = (new(x["q"].shape, dtype=x["q"].dtype, device="cuda"), new(x["k"].shape, dtype=x["k"].dtype, device="cuda"))
        else:
            s["out"] = (torch.empty_like(x["dq"]), torch.empty_like(x["dk"]))
        if c["op"] == "norm_grad":
            s["dw"] = (new(c["d"], device="cuda"), new(c["d"], device="cuda"))
        if own:
            from chunk_scheduled_communication_gb300 import rope
            s["plan"] = rope.RopePlan(d=c["d"], d_rot=c["rot"], layout=c["layout"], base=BASE, scaling=_scaling(c),
                                      dtype=c["dtype"])
        else:
            # the cosines and sines of every position, as models keep them
            f, factor = _frequencies(c)
            turn = torch.arange(c["max_pos"], dtype=torch.float64, device="cuda")[:, None] * f.cuda()
            s["cos"], s["sin"] = (turn.cos() * factor).float(), (turn.sin() * factor).float()
        return s
    if c["op"] == "decode":
        s["out"] = torch.empty_like(x["q"])
        if own:
            from chunk_scheduled_communication_gb300 import window
            s["plan"] = window.DecodePlan(max_seqs=c["batch"], H_q=c["hq"], H_kv=c["hkv"], d=c["d"], window=c["window"],
                                          sinks=c["sinks"], page_size=c["page"], dtype=c["dtype"])
        return s
    q_lens, k_lens = _lens(c, "q_lens"), _lens(c, "k_lens")
    s["out"] = torch.empty_like(x["q"])
    if c["op"] == "window_train":
        s["lse"] = new(x["q"].shape[:2], device="cuda")
        s["grads"] = tuple(torch.empty_like(x[n]) for n in "qkv")
    if own:
        from chunk_scheduled_communication_gb300 import window
        s["plan"] = window.WindowPlan(q_lens, k_lens, H_q=c["hq"], H_kv=c["hkv"], d=c["d"], window=c["window"],
                                      sinks=c["sinks"], dtype=c["dtype"], backward=c["op"] == "window_train")
    else:
        s["rows"] = _row_blocks(c, q_lens, k_lens)
    return s


def _row_blocks(case, q_lens, k_lens):
    """Blocks of BLOCK query rows and the keys they may see: query rows, key rows, and both positions
    (-1: none), which tell the plain form where to read."""
    window, sinks = case["window"], case["sinks"]
    size = min(BLOCK, max(max(q_lens), 1))
    most = min(window + size - 1 + sinks, max(max(k_lens), 1))
    q_row, q_pos, k_row, k_pos = [], [], [], []
    q0 = k0 = 0
    for ql, kl in zip(q_lens, k_lens):
        for i in range(0, ql, size):
            r = torch.arange(i, i + size)
            p = torch.where(r < ql, r + kl - ql, -1)
            q_row.append(torch.where(r < ql, r + q0, -1))
            q_pos.append(p)
            first, last = max(i + kl - ql, 0), min(i + size, ql) + kl - ql
            lo = max(first - window + 1, 0)
            j = torch.cat([torch.arange(0, min(sinks, lo)), torch.arange(lo, max(last, lo))])[:most]
            j = torch.cat([j, torch.full((most - j.numel(),), -1)])
            k_row.append(torch.where(j >= 0, j + k0, -1))
            k_pos.append(j)
        q0, k0 = q0 + ql, k0 + kl
    return [torch.stack(t).cuda() for t in (q_row, q_pos, k_row, k_pos)]


# ---------------------------------------------------------------------------------------- plain forms
def _turn(x, cos, sin, rot, interleaved):
    """The rotation of the last axis's first `rot` elements by tables [tokens, rot/2]."""
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_heads(s):
    c = s["case"]
    cos, sin = s["cos"][s["pos"]], s["sin"][s["pos"]]
    inter = c["layout"] == "interleaved"
    if c["op"] == "rope":
        return tuple(_turn(s[n].float(), cos, sin, c["rot"], inter).to(s[n].dtype) for n in "qk")
    if c["op"] == "rope_grad":
        return tuple(_turn(s[n].float(), cos, -sin, c["rot"], inter).to(s[n].dtype) for n in ("dq", "dk"))

    def norm(n):
        x, w = s[n].float(), s["w" + n].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return _turn(x * r * w, cos, sin, c["rot"], inter).to(s[n].dtype)

    def grad(n):
        x, w = s[n].float(), s["w" + n].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        y = _turn(s["d" + n].float(), cos, -sin, c["rot"], inter)
        h = x * r
        dx = r * (y * w - h * (y * w * h).mean(-1, keepdim=True))
        return dx.to(s[n].dtype), (y * h).sum((0, 1))

    if c["op"] == "norm":
        return norm("q"), norm("k")
    (dq, dwq), (dk, dwk) = grad("q"), grad("k")
    return dq, dk, dwq, dwk


def _plain_attention(c, q, k, v, rows, do=None):
    q_row, q_pos, k_row, k_pos = rows
    group, scale = c["hq"] // c["hkv"], c["d"] ** -0.5

    def split(x):  # [blocks, rows, heads, d] -> [blocks, kv heads, group, rows, d]
        b, n, h, d = x.shape
        return x.view(b, n, c["hkv"], h // c["hkv"], d).permute(0, 2, 3, 1, 4)

    def join(x):
        b, _, _, n, d = x.shape
        return x.permute(0, 3, 1, 2, 4).reshape(b * n, -1, d)

    def flat(x):  # the group's rows as one axis
        return x.reshape(*x.shape[:2], -1, x.shape[-1])

    qb = flat(split(q.float()[q_row]))
    kb, vb = split(k.float()[k_row])[:, :, 0], split(v.float()[k_row])[:, :, 0]
    p, j = q_pos[:, :, None], k_pos[:, None, :]
    seen = (p >= 0) & (j >= 0) & (j <= p) & ((j > p - c["window"]) | (j < c["sinks"]))
    seen = seen[:, None, None].expand(-1, 1, group, -1, -1).flatten(2, 3)
    a = (qb @ kb.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = a.amax(-1, keepdim=True)
    a = a.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = a.sum(-1, keepdim=True)
    a = a.div_(total.masked_fill(total == 0, 1.0))

    def shape(x):  # back to [blocks, kv heads, group, rows, d]
        return x.view(*x.shape[:2], group, -1, x.shape[-1])

    out = torch.zeros(q.shape[0] + 1, *q.shape[1:], device=q.device)
    out[q_row.flatten()] = join(shape(a @ vb))
    if do is None:
        return out[:-1].to(q.dtype)
    dob = flat(split(do.float()[q_row]))
    dv = torch.zeros(k.shape[0] + 1, *k.shape[1:], device=q.device)
    dk, dq = torch.zeros_like(dv), torch.zeros_like(out)
    dv.index_add_(0, k_row.flatten().remainder(k.shape[0] + 1), join((a.transpose(-1, -2) @ dob)[:, :, None]))
    da = dob @ vb.transpose(-1, -2)
    da = da.sub_((a * da).sum(-1, keepdim=True)).mul_(a).mul_(scale)
    dq[q_row.flatten()] = join(shape(da @ kb))
    dk.index_add_(0, k_row.flatten().remainder(k.shape[0] + 1), join((da.transpose(-1, -2) @ qb)[:, :, None]))
    return out[:-1].to(q.dtype), dq[:-1].to(q.dtype), dk[:-1].to(k.dtype), dv[:-1].to(v.dtype)


def _plain_decode(s):
    c, lens = s["case"], s["lens"].long()
    lo = (lens - c["window"]).clamp(min=0)[:, None]
    n = min(c["window"] + c["sinks"], c["max_len"])
    i = torch.arange(n, device="cuda")[None]
    first = lo.clamp(max=c["sinks"])
    j = torch.where(i < first, i, lo + i - first)
    j = torch.where(j < lens[:, None], j, -1)
    page = s["table"].long().gather(1, j.clamp(min=0) // c["page"])
    row = torch.where(j >= 0, page * c["page"] + j.clamp(min=0) % c["page"], -1)
    at = torch.arange(c["batch"], device="cuda")[:, None]
    return _plain_attention(c, s["q"], s["k"].flatten(0, 1), s["v"].flatten(0, 1), (at, lens[:, None] - 1, row, j))


def run(state):
    s, c = state, state["case"]
    if not own:
        if "tokens" in c:
            return _plain_heads(s)
        if c["op"] == "decode":
            return _plain_decode(s)
        return _plain_attention(c, s["q"], s["k"], s["v"], s["rows"], s.get("do"))
    plan = s["plan"]
    if c["op"] == "rope":
        plan.rotate(s["q"], s["out"][0], s["k"], s["out"][1], positions=s["pos"])
    elif c["op"] == "rope_grad":
        plan.rotate_backward(s["dq"], s["out"][0], s["dk"], s["out"][1], positions=s["pos"])
    elif c["op"] == "norm":
        plan.norm_rotate(s["q"], s["out"][0], s["wq"], s["k"], s["out"][1], s["wk"], positions=s["pos"], eps=EPS)
    elif c["op"] == "norm_grad":
        plan.norm_rotate_backward(s["q"], s["dq"], s["out"][0], s["wq"], s["dw"][0], s["k"], s["dk"], s["out"][1],
                                  s["wk"], s["dw"][1], positions=s["pos"], eps=EPS)
        return s["out"] + s["dw"]
    elif c["op"] == "decode":
        plan.run(s["q"], s["k"], s["v"], s["lens"], s["out"], page_table=s["table"])
    elif c["op"] == "window":
        plan.forward(s["q"], s["k"], s["v"], s["out"])
    else:
        plan.forward(s["q"], s["k"], s["v"], s["out"], lse=s["lse"])
        plan.backward(s["do"], s["q"], s["k"], s["v"], s["out"], s["lse"], *s["grads"])
        return (s["out"],) + s["grads"]
    return s["out"]


# ---------------------------------------------------------------------------------------- 64 bits
def _exact_heads(c, x):
    f, factor = _frequencies(c)
    turn = x["pos"].double()[:, None, None] * f.cuda()
    cs = torch.polar(torch.full_like(turn, factor), turn)
    rot, half = c["rot"], c["rot"] // 2
    first = torch.arange(half) * 2 if c["layout"] == "interleaved" else torch.arange(half)
    second = first + (1 if c["layout"] == "interleaved" else half)

    def turned(t, by):  # each pair as a complex number
        y = t.clone()
        z = torch.complex(t[..., first], t[..., second]) * by
        y[..., first], y[..., second] = z.real, z.imag
        return y

    if c["op"] == "rope":
        return tuple(turned(x[n].double(), cs) for n in "qk")
    if c["op"] == "rope_grad":
        return tuple(turned(x[n].double(), cs.conj()) for n in ("dq", "dk"))
    out, dw = [], []
    for n in "qk":
        t, w = x[n].double(), x["w" + n].double()
        r = 1 / torch.sqrt(t.square().sum(-1, keepdim=True) / c["d"] + EPS)
        if c["op"] == "norm":
            out.append(turned(t * r * w, cs))
            continue
        y = turned(x["d" + n].double(), cs.conj())
        dw.append((y * t * r).sum((0, 1)))
        y = y * w
        out.append(r * y - t * r ** 3 * (y * t).sum(-1, keepdim=True) / c["d"])
    return tuple(out + dw)


def _exact_attention(c, x):
    """Sequence by sequence, kv head by kv head, over whole rows of scores."""
    q, k, v = (x[n].double() for n in "qkv")
    do = x["do"].double() if "do" in x else None
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    group, scale = c["hq"] // c["hkv"], 1 / math.sqrt(c["d"])
    q0 = k0 = 0
    for ql, kl in zip(_lens(c, "q_lens"), _lens(c, "k_lens")):
        for i in range(0, ql, 1024):
            n = min(1024, ql - i)
            p = torch.arange(i + kl - ql, i + n + kl - ql, device="cuda")[:, None]
            end = int(p[-1]) + 1
            if end <= 0:
                continue
            mid = min(max(int(p[0]) - c["window"] + 1, 0), end)
            j = torch.cat([torch.arange(min(c["sinks"], mid), device="cuda"), torch.arange(mid, end, device="cuda")])
            hidden = (j > p) | ((j <= p - c["window"]) & (j >= c["sinks"]))
            some = (~hidden).any(-1, keepdim=True)
            for h in range(c["hq"]):
                g = h // group
                rows = slice(q0 + i, q0 + i + n)
                kk, vv = k[k0 + j, g], v[k0 + j, g]
                s = (q[rows, h] @ kk.T * scale).masked_fill(hidden, -math.inf)
                w = torch.softmax(s.masked_fill(~some, 0.0), -1) * some * ~hidden
                o[rows, h] = w @ vv
                if do is not None:
                    dw = do[rows, h] @ vv.T
                    ds = w * (dw - (do[rows, h] * o[rows, h]).sum(-1, keepdim=True)) * scale
                    dq[rows, h] = ds @ kk
                    dk[:, g].index_add_(0, k0 + j, ds.T @ q[rows, h])
                    dv[:, g].index_add_(0, k0 + j, w.T @ do[rows, h])
        q0, k0 = q0 + ql, k0 + kl
    return o if do is None else (o, dq, dk, dv)


def _exact_decode(c, x):
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_decode_lens(c, 0)):
        j = torch.arange(n, device="cuda")
        j = j[(j >= n - c["window"]) | (j < c["sinks"])]
        page = x["table"][b].long()[j // c["page"]]
        k, v = x["k"][page, j % c["page"]].double(), x["v"][page, j % c["page"]].double()
        q = x["q"][b].double().view(c["hkv"], -1, c["d"])
        w = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(c["d"]), -1)
        out[b] = torch.einsum("hgn,nhd->hgd", w, v).reshape(c["hq"], c["d"])
    return out


def exact(case, seed):
    x = _inputs(case, seed)
    if "tokens" in case:
        return _exact_heads(case, x)
    return _exact_decode(case, x) if case["op"] == "decode" else _exact_attention(case, x)
