"""The operators of a decoder layer's halves in training and serving: the attention
half (head norm and rotation, windowed attention with sinks, their gradients,
decoding over a paged cache) and the feed-forward half (layer norm, gated block,
their gradients), with the clipping of all their gradients.  The output and down
projections and the residual sums of a whole layer are not part of it: the
attention's rows go into the layer norm as they are.

    python -m chunk_scheduled_communication_gb300.window_layer --tokens 1000 --new 16

runs a training step of the attention on a packed batch, then a prompt with
``--new`` decoding steps, checks the decoded rows against the same rows of one
long prompt, runs a training step of both halves, and prints the times (CUDA
events, no L2 flush: not a benchmark).

A projection gives ``qkv`` rows of ``H_q + 2 H_kv`` heads; the layer reads it in
place through strides and returns the gradient in the same form."""
from __future__ import annotations

import argparse

import torch

from . import clip, ffn, norm, rope, window

NORM_MOST = 16384  # elements of a row that the layer norm takes (include/syn_norm.h)


class WindowLayer:
    """Norm, rotation and windowed attention with the same weights for training,
    prompts and decoding."""

    def __init__(self, H_q, H_kv, d, window, sinks, base=10000.0, scaling=None, eps=1e-6, dtype="bf16"):
        self.H_q, self.H_kv, self.d, self.window, self.sinks = H_q, H_kv, d, window, sinks
        self.eps, self.dtype, self.type = eps, dtype, rope.torch_dtype(dtype)
        self.rope = rope.RopePlan(d=d, base=base, scaling=scaling, dtype=dtype)
        self.wq = torch.ones(d, dtype=self.type, device="cuda")
        self.wk = torch.ones(d, dtype=self.type, device="cuda")

    def plan(self, lens, backward=False):
        """The attention plan of a packed batch of sequences."""
        return window.WindowPlan(lens, H_q=self.H_q, H_kv=self.H_kv, d=self.d, window=self.window, sinks=self.sinks,
                                 dtype=self.dtype, backward=backward)

    def split(self, qkv):
        a, b = self.H_q, self.H_q + self.H_kv
        return qkv[:, :a], qkv[:, a:b], qkv[:, b:]

    def forward(self, plan, qkv, positions):
        """The output rows [tokens, H_q, d], and what backward needs."""
        q, k, v = self.split(qkv)
        qr, kr = torch.empty(q.shape, dtype=self.type, device="cuda"), torch.empty(k.shape, dtype=self.type, device="cuda")
        self.rope.norm_rotate(q, qr, self.wq, k, kr, self.wk, positions=positions, eps=self.eps)
        out, lse = torch.empty_like(qr), torch.empty(qr.shape[:2], device="cuda")
        plan.forward(qr, kr, v, out, lse=lse)
        return out, (qkv, qr, kr, out, lse, positions)

    def backward(self, plan, saved, d_out):
        """The gradients of qkv and of the two norm weights (fp32)."""
        qkv, qr, kr, out, lse, positions = saved
        q, k, v = self.split(qkv)
        d_qkv = torch.empty_like(qkv)
        dq, dk, dv = self.split(d_qkv)
        plan.backward(d_out, qr, kr, v, out, lse, dq, dk, dv)
        dwq, dwk = torch.empty(self.d, device="cuda"), torch.empty(self.d, device="cuda")
        # in place: the rotated heads' gradients become the projection's
        self.rope.norm_rotate_backward(q, dq, dq, self.wq, dwq, k, dk, dk, self.wk, dwk, positions=positions, eps=self.eps)
        return d_qkv, dwq, dwk


class FeedForward:
    """Layer norm and gated block with the same weights for training and serving.  Training
    keeps the block's projections in fp32 (its gradients' errors are 1.4 times a single
    rounding's then; 1.8 with projections of the rows' type)."""

    def __init__(self, d, d_ff, act="silu", eps=1e-5, dtype="bf16", seed=1):
        self.eps, self.type = eps, rope.torch_dtype(dtype)
        self.norm, self.ffn = norm.NormPlan(d=d, dtype=dtype), ffn.FfnPlan(d=d, d_ff=d_ff, act=act, dtype=dtype, saved="fp32")
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.w = torch.ones(d, dtype=self.type, device="cuda")
        self.b = torch.zeros(d, dtype=self.type, device="cuda")
        self.wg, self.wu = ((torch.randn(d, d_ff, generator=g, device="cuda") * d ** -0.5).to(self.type) for _ in range(2))

    def forward(self, x, train=True):
        """The rows [tokens, d_ff] in front of the down projection, and what backward needs."""
        y = torch.empty_like(x)
        self.norm.forward(x, y, self.w, self.b, eps=self.eps)
        h, g, u = (torch.empty(x.shape[0], self.wg.shape[1], dtype=t, device="cuda") if wanted else None
                   for t, wanted in ((self.type, True), (self.ffn.saved, train), (self.ffn.saved, train)))
        self.ffn.forward(y, self.wg, self.wu, h, G=g, U=u)
        return h, (x, y, g, u)

    def backward(self, saved, d_h):
        """The gradient of x and those of the weights w, b (fp32), wg and wu."""
        x, y, g, u = saved
        dwg, dwu, dx = torch.empty_like(self.wg), torch.empty_like(self.wu), torch.empty_like(x)
        dw, db = torch.empty(x.shape[1], device="cuda"), torch.empty(x.shape[1], device="cuda")
        dg, du = torch.empty_like(d_h), torch.empty_like(d_h)
        self.ffn.backward(d_h, y, self.wg, self.wu, g, u, dg, du, dx, dwg, dwu)
        self.norm.backward(x, dx, dx, self.w, dw, db, eps=self.eps)
        return dx, [dw, db, dwg, dwu]


def train_step(layer, feed, clipping, plan, qkv, positions, d_h, max_norm):
    """One training step of both halves, the attention's rows going into the layer norm as
    they are: the feed-forward half's rows, the gradient of qkv, the weights' gradients (of the head norms, the layer norm's w and b, the
    block's wg and wu) clipped in place, and their norm."""
    out, saved = layer.forward(plan, qkv, positions)
    h, kept = feed.forward(out.flatten(1))
    d_out, grads = feed.backward(kept, d_h)
    d_qkv, dwq, dwk = layer.backward(plan, saved, d_out.view_as(out))
    grads, total = [dwq, dwk] + grads, torch.empty(1, device="cuda")
    clipping.clip(grads, max_norm, total)
    return h, d_qkv, grads, total


class PagedCache:
    """K and V pages of a batch of sequences, page after page as they grow."""

    def __init__(self, layer, n_seqs, max_len, page=64):
        per = (max_len + page - 1) // page
        shape = (n_seqs * per, page, layer.H_kv, layer.d)
        self.page, self.max_len, self.longest = page, per * page, 0
        self.k = torch.empty(shape, dtype=layer.type, device="cuda")
        self.v = torch.empty(shape, dtype=layer.type, device="cuda")
        self.table = torch.arange(n_seqs * per, dtype=torch.int32, device="cuda").view(n_seqs, per)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.plan = window.DecodePlan(max_seqs=n_seqs, H_q=layer.H_q, H_kv=layer.H_kv, d=layer.d, window=layer.window,
                                      sinks=layer.sinks, page_size=page, dtype=layer.dtype)

    def rows(self):
        """K and V as rows that `slots` index."""
        return self.k.flatten(0, 1), self.v.flatten(0, 1)

    def grow(self, longest):
        """The longest sequence is to have so many tokens (known to the host:
        positions past the table would index out of it on the device)."""
        if longest > self.max_len:
            raise ValueError(f"a sequence of {longest} tokens in a cache of {self.max_len} a sequence")
        self.longest = longest

    def slots(self, seq, pos):
        """Cache rows of positions `pos` of sequences `seq` (int64)."""
        return self.table[seq, pos // self.page].long() * self.page + pos % self.page


def prompt(layer, plan, cache, qkv, lens):
    """The outputs of a packed batch of prompts; their K and V go to the cache."""
    if len(lens) != cache.lens.shape[0]:
        raise ValueError(f"{len(lens)} prompts for a cache of {cache.lens.shape[0]} sequences")
    cache.grow(max(lens))
    n = torch.tensor(lens, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n)
    pos = torch.cat([torch.arange(x, device="cuda") for x in lens])
    q, k, v = layer.split(qkv)
    qr, kr = torch.empty(q.shape, dtype=layer.type, device="cuda"), torch.empty(k.shape, dtype=layer.type, device="cuda")
    layer.rope.norm_rotate(q, qr, layer.wq, k, kr, layer.wk, positions=pos, eps=layer.eps)
    ck, cv = cache.rows()
    slots = cache.slots(seq, pos)
    ck[slots], cv[slots] = kr, v
    cache.lens.copy_(n)
    out = torch.empty_like(qr)
    plan.forward(qr, kr, v, out)
    return out


def decode(layer, cache, qkv):
    """One new token per sequence: its K (normed and rotated) and V are written
    into the cache in the pass that makes its query, then attended."""
    cache.grow(cache.longest + 1)
    pos = cache.lens.long()
    q, k, v = layer.split(qkv)
    qr, out = torch.empty(q.shape, dtype=layer.type, device="cuda"), torch.empty(q.shape, dtype=layer.type, device="cuda")
    ck, cv = cache.rows()
    slots = cache.slots(torch.arange(qkv.shape[0], device="cuda"), pos)
    layer.rope.norm_rotate(q, qr, layer.wq, k, ck, layer.wk, v, cv, positions=pos, eps=layer.eps, slots=slots)
    cache.lens += 1
    cache.plan.run(qr, cache.k, cache.v, cache.lens, out, page_table=cache.table)
    return out


def _timed(f):
    e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    e[0].record()
    r = f()
    e[1].record()
    torch.cuda.synchronize()
    return r, e[0].elapsed_time(e[1])


def run(tokens=1000, new=16, H_q=8, H_kv=2, d=128, width=256, sinks=4, seed=0, d_ff=1024, max_norm=1.0):
    """A training step of the attention, a prompt with decoding, and a training step
    of both halves (None where the heads make rows wider than the layer norm takes);
    returns a dict of what was computed and the largest difference between decoding
    and one long prompt."""
    torch.cuda.set_device(0)
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer = WindowLayer(H_q, H_kv, d, width, sinks)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(layer.type)
    lens = [tokens, max(tokens // 3, 1)]
    total = sum(lens)
    qkv, d_out = draw(total, H_q + 2 * H_kv, d), draw(total, H_q, d)
    positions = torch.cat([torch.arange(n, device="cuda") for n in lens])
    plan = layer.plan(lens, backward=True)
    (out, saved), ms_f = _timed(lambda: layer.forward(plan, qkv, positions))
    (d_qkv, dwq, dwk), ms_b = _timed(lambda: layer.backward(plan, saved, d_out))
    plan.check()
    # prompts of all but the last `new` tokens, the rest one by one
    first = [max(n - new, 0) for n in lens]
    keep = torch.cat([torch.arange(o, o + f) for o, f in zip((0, lens[0]), first)]).cuda()
    cache = PagedCache(layer, 2, max(lens))
    head = prompt(layer, layer.plan(first), cache, qkv[keep], first)
    worst = (head.float() - out[keep].float()).abs().max().item() if len(keep) else 0.0
    steps = min(n - f for n, f in zip(lens, first))
    ms_d = 0.0
    for i in range(steps):
        at = torch.tensor([first[0] + i, lens[0] + first[1] + i], device="cuda")
        o, ms = _timed(lambda: decode(layer, cache, qkv[at]))
        ms_d += ms
        worst = max(worst, (o.float() - out[at].float()).abs().max().item())
    cache.plan.check()
    ms = {"forward": ms_f, "backward": ms_b, "decode_step": ms_d / max(steps, 1)}
    step = None
    if H_q * d <= NORM_MOST:
        # both halves: the gradient of the feed-forward half's rows is given
        feed, clipping = FeedForward(H_q * d, d_ff), clip.ClipPlan()
        d_h = draw(total, d_ff)
        (h, d_both, grads, norm_), ms["step"] = _timed(
            lambda: train_step(layer, feed, clipping, plan, qkv, positions, d_h, max_norm))
        feed.ffn.check()
        plan.check()
        step = {"h": h, "d_h": d_h, "d_qkv": d_both, "grads": grads, "norm": norm_, "feed": feed, "max_norm": max_norm}
    return {"step": step, "out": out, "d_qkv": d_qkv, "dwq": dwq, "dwk": dwk, "qkv": qkv, "d_out": d_out, "positions": positions,
            "lens": lens, "layer": layer, "worst": worst, "v_max": qkv[:, H_q + H_kv:].abs().max().item(), "ms": ms}


def main():
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--tokens", type=int, default=1000)
    a.add_argument("--new", type=int, default=16)
    a.add_argument("--heads", type=int, nargs=2, default=(8, 2), metavar=("H_q", "H_kv"))
    a.add_argument("--window", type=int, default=256)
    a.add_argument("--sinks", type=int, default=4)
    a.add_argument("--d-ff", type=int, default=1024)
    o = a.parse_args()
    r = run(o.tokens, o.new, *o.heads, width=o.window, sinks=o.sinks, d_ff=o.d_ff)
    ms, step = r["ms"], r["step"]
    print("attention forward %.3f ms, backward %.3f ms, decoding step %.3f ms; decoding against the prompt: at most %.2e apart"
          % (ms["forward"], ms["backward"], ms["decode_step"], r["worst"]))
    if step is not None:
        print("training step of both halves %.3f ms; gradient norm %.3f" % (ms["step"], step["norm"].item()))


if __name__ == "__main__":
    main()
