"""The operators together, as chunk_scheduled_communication_gb300/window_layer.py
uses them: a training step against a plain implementation in 64 bits with
automatic differentiation, and decoding against one long prompt.

Tolerance, u = 2^-8 (bf16): Q and K are rounded after norm and rotation, the
probabilities and score gradients before their products, O, dQ and dK after
theirs, and dqkv once more.  Each rounding is at most u of its value, half of
that and random in its mean; relative to the norm of the whole tensor the
output takes three (q, k in the scores, p, o) and the gradients six:
4 u and 8 u.
"""
import math

import pytest
import torch

from chunk_scheduled_communication_gb300 import syn, window_layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    syn.lib()


def plain(layer, qkv, wq, wk, positions, lens):
    f = 10000.0 ** (-torch.arange(0, layer.d, 2, dtype=torch.float64, device="cuda") / layer.d)
    ang = positions.double()[:, None, None] * f

    def head(x, w):
        h = x / torch.sqrt((x * x).mean(-1, keepdim=True) + layer.eps) * w
        a, b = h[..., :layer.d // 2], h[..., layer.d // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1)

    q, k, v = layer.split(qkv)
    q, k = head(q, wq), head(k, wk)
    g, out, at = layer.H_q // layer.H_kv, [], 0
    for n in lens:
        p = torch.arange(n, device="cuda")
        see = (p[None] <= p[:, None]) & ((p[None] > p[:, None] - layer.window) | (p[None] < layer.sinks))
        qq, kk, vv = (t[at:at + n].transpose(0, 1) for t in (q, k, v))
        s = qq @ kk.repeat_interleave(g, 0).transpose(1, 2) / math.sqrt(layer.d)
        out.append((torch.softmax(s.masked_fill(~see, -math.inf), -1) @ vv.repeat_interleave(g, 0)).transpose(0, 1))
        at += n
    return torch.cat(out)


def test_training_step_and_decoding():
    r = window_layer.run(tokens=400, new=9, H_q=4, H_kv=2, width=90, sinks=3)
    layer = r["layer"]
    x = r["qkv"].double().requires_grad_()
    wq, wk = layer.wq.double().requires_grad_(), layer.wk.double().requires_grad_()
    ref = plain(layer, x, wq, wk, r["positions"], r["lens"])
    (ref * r["d_out"].double()).sum().backward()

    def off(a, b):
        return ((a.double() - b).norm() / b.norm()).item()

    assert off(r["out"], ref.detach()) <= 4 * U
    assert off(r["d_qkv"], x.grad) <= 8 * U
    assert off(r["dwq"], wq.grad) <= 8 * U and off(r["dwk"], wk.grad) <= 8 * U
    # two ways to the same rows: each within (2 u + 2^-14) of max|v|
    assert r["worst"] <= 2 * (2 * U + 2.0 ** -14) * r["v_max"]


def test_a_cache_that_is_full():
    """Refused on the host, before any position indexes past the page table."""
    layer = window_layer.WindowLayer(2, 1, 64, 16, 2)
    cache = window_layer.PagedCache(layer, 2, 20, page=8)  # 24 tokens a sequence
    rows = lambda n: torch.randn(n, 4, 64, device="cuda").bfloat16()
    for bad in ([25, 3], [3], [1, 2, 3]):
        with pytest.raises(ValueError):
            window_layer.prompt(layer, layer.plan(bad), cache, rows(sum(bad)), bad)
    window_layer.prompt(layer, layer.plan([22, 3]), cache, rows(25), [22, 3])
    for _ in range(2):
        window_layer.decode(layer, cache, rows(2))
    before = cache.k.clone()
    with pytest.raises(ValueError):
        window_layer.decode(layer, cache, rows(2))
    cache.plan.check()
    assert cache.lens.tolist() == [24, 5] and torch.equal(cache.k.nan_to_num(), before.nan_to_num())
