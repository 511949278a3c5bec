"""A training step of a decoder layer's two halves, as
chunk_scheduled_communication_gb300/window_layer.py runs it, against a plain
implementation in 64 bits with automatic differentiation.

Tolerance, u = 2^-8 (bf16): relative to the norm of the whole tensor each rounding on
the way counts u (at most u of its value, half of that and random in its mean).  The
rows h take the rotated heads (in the scores), the probabilities, the attention's
output, the norm's output, and h's own: 6 u.  A gradient takes besides these
roundings of its operands G and U (through slopes up to 1.13), dG and dU, the block's dX,
the norm's dX, and the attention's and the head norms' (8 u, as tests/test_gpu_window_layer.py
counts them): 18 u.
"""
import math

import pytest
import torch

from chunk_scheduled_communication_gb300 import syn, window_layer
from test_gpu_window_layer import plain

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    syn.lib()


@pytest.mark.parametrize("tokens, d_ff, max_norm", [(400, 640, 1.0), (77, 1032, 1e9)])
def test_training_step(tokens, d_ff, max_norm):
    r = window_layer.run(tokens=tokens, new=2, H_q=4, H_kv=2, width=90, sinks=3, d_ff=d_ff, max_norm=max_norm)
    layer, s = r["layer"], r["step"]
    feed = s["feed"]
    leaves = [t.double().requires_grad_() for t in (r["qkv"], layer.wq, layer.wk, feed.w, feed.b, feed.wg, feed.wu)]
    x, wq, wk, w, b, wg, wu = leaves
    rows = plain(layer, x, wq, wk, r["positions"], r["lens"]).flatten(1)
    var, mean = torch.var_mean(rows, -1, unbiased=False, keepdim=True)
    y = (rows - mean) / torch.sqrt(var + feed.eps) * w + b
    h = torch.nn.functional.silu(y @ wg) * (y @ wu)
    grads = torch.autograd.grad(h, leaves, s["d_h"].double())
    off = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    assert off(s["h"], h.detach()) <= 6 * U
    assert off(s["d_qkv"], grads[0]) <= 18 * U
    norm = math.sqrt(sum(float((g * g).sum()) for g in grads[1:]))
    assert abs(s["norm"].item() - norm) <= 18 * U * norm
    c = min(1.0, max_norm / (s["norm"].item() + 1e-6))
    for got, want in zip(s["grads"], grads[1:]):
        assert off(got, want * c) <= 18 * U
    clipped = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"]))
    assert abs(clipped - min(max_norm, s["norm"].item())) <= U * clipped


def test_serving_gives_the_rows_of_training():
    feed = window_layer.FeedForward(512, 768, act="gelu_tanh", dtype="fp16")
    x = torch.randn(33, 512, device="cuda").half()
    h, saved = feed.forward(x)
    served, none = feed.forward(x, train=False)
    assert torch.equal(h, served) and none[2] is None and saved[2] is not None


def test_a_step_in_a_graph():
    """The same bits as the eager step's, for new inputs in the graph's buffers."""
    layer, feed = window_layer.WindowLayer(4, 2, 64, 50, 2), window_layer.FeedForward(256, 384)
    clipping = window_layer.clip.ClipPlan()
    lens = [150, 61]
    plan = layer.plan(lens, backward=True)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    qkv, d_h = torch.empty(211, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(211, 384, dtype=torch.bfloat16, device="cuda")
    step = lambda: window_layer.train_step(layer, feed, clipping, plan, qkv, pos, d_h, 1.0)

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        d_h.copy_(torch.randn(d_h.shape, generator=g, device="cuda"))

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, d_qkv, grads, norm = step()
    for seed in (1, 2, 1):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, d_qkv, norm, *grads)]
        a, b, c, e = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (a, b, e, *c)))
    plan.check()
    feed.ffn.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_layer_keeps_its_projections_in_fp32(dtype):
    """The weights' gradients of the block against those of its own input in 64 bits.  dG (or
    dU) and the result are rounded once each, with errors of random signs, so that their
    squares add: relative to the norm the error is the root of the sum of both roundings'
    squares, as the 64-bit values' own roundings give them (over 100000 elements: to 1 %;
    1.1 is allowed).  Projections rounded to 16 bits would give 1.24 to 1.33 of it."""
    feed = window_layer.FeedForward(512, 768, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, d_h = (torch.randn(600, c, generator=g, device="cuda").to(feed.type) for c in (512, 768))
    h, saved = feed.forward(x)
    y = saved[1]
    grads = feed.backward(saved, d_h)[1]
    feed.ffn.check()
    wg, wu = feed.wg.double().requires_grad_(), feed.wu.double().requires_grad_()
    a, b = y.double() @ wg, y.double() @ wu
    want = torch.autograd.grad(torch.nn.functional.silu(a) * b, [a, b, wg, wu], d_h.double())
    step = lambda t: ((t.to(feed.type).double() - t).norm() / t.norm()).item()
    for got, inner, ref in zip(grads[2:], want[:2], want[2:]):
        error = ((got.double() - ref).norm() / ref.norm()).item()
        assert error <= 1.1 * math.hypot(step(inner), step(ref))


def test_heads_that_make_rows_wider_than_the_norm_takes():
    """The attention half runs all the same."""
    r = window_layer.run(tokens=70, new=2, H_q=132, H_kv=4, width=40, sinks=2)
    assert r["step"] is None and "step" not in r["ms"]
    assert r["out"].shape[1:] == (132, 128) and all(r[k].isfinite().all() for k in ("out", "d_qkv", "dwq", "dwk"))
    assert r["worst"] <= (2.0 ** -6 + 2.0 ** -13) * r["v_max"]
