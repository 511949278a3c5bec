"""GPU parity of the rotary positions and the head norm with rotation
(include/syn_rope.h) against plain 64-bit implementations, through the C ABI.

Tolerances, from the kernels' arithmetic: a value computed in fp32, within a
bound of the 64-bit one, is rounded once to the type, so the result lies
between the roundings of the bound's two ends.  The rotation takes an angle right to 2^-23 radians, a sine and a cosine within
2 ulp, two products and a sum: under 16 * 2^-24 of |a| + |b|.  The norm adds a
sum of up to 256 squares over at most 16 terms a lane and 5 levels of lanes,
its root within 2 ulp and three products: under 64 * 2^-24 in all.  A weight
gradient sums n rows of fp32 products in chains: under (n + 128) * 2^-24 of
the sum of their magnitudes.
"""
import math

import numpy as np
import pytest
import torch

from chunk_scheduled_communication_gb300 import rope, syn

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24
SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="ntk", factor=8.0),
            dict(kind="llama3", factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original_context=8192),
            dict(kind="yarn", factor=4.0, original_context=32768, beta_fast=32.0, beta_slow=1.0)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    syn.lib()


def frequencies(rot, base, s):
    i = np.arange(rot // 2, dtype=np.float64)
    kind = s["kind"] if s else "none"
    if kind == "ntk":
        base = base * s["factor"] ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if kind == "linear":
        return f / s["factor"], 1.0
    if kind == "llama3":
        out = []
        for v in f:
            wave = 2 * math.pi / v
            if wave <= s["original_context"] / s["high_freq_factor"]:
                out.append(v)
            elif wave >= s["original_context"] / s["low_freq_factor"]:
                out.append(v / s["factor"])
            else:
                t = (s["original_context"] / wave - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])
                out.append((1 - t) * v / s["factor"] + t * v)
        return np.array(out), 1.0
    if kind == "yarn":
        n = lambda t: rot * math.log(s["original_context"] / (t * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(n(s["beta_fast"])), 0), min(math.ceil(n(s["beta_slow"])), rot - 1)
        r = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - r) + f / s["factor"] * r, 0.1 * math.log(s["factor"]) + 1
    return f, 1.0


def pairs(rot, layout):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)


def turn(x, pos, rot, layout, f, factor, sign=1):
    """R(pos) x of [t, h, d] in 64 bits, and |a| + |b| of each element's pair."""
    y, mag = x.copy(), np.abs(x)
    a, b = pairs(rot, layout)
    ang = pos.astype(np.float64)[:, None, None] * f
    c, s = factor * np.cos(ang), sign * factor * np.sin(ang)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    m = factor * (mag[..., a] + mag[..., b])
    mag = mag.copy()
    mag[..., a], mag[..., b] = m, m
    return y, mag


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, ref, tol):
    """got is the rounding to its type of a value within tol of ref."""
    lo, hi = (f64(torch.from_numpy(ref + s * tol).to(got.dtype)) for s in (-1, 1))
    got = f64(got)
    assert ((lo <= got) & (got <= hi)).all(), float(np.maximum(lo - got, got - hi).max())


def make(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(TYPES[dtype]).cuda()


SHAPES = [  # tokens, hq, hkv, d, rot
    (1, 1, 1, 128, 128), (3, 32, 8, 128, 64), (257, 7, 1, 64, 64), (5, 4, 4, 256, 256), (33, 3, 2, 80, 48),
    (2, 2, 1, 6, 4), (9, 5, 3, 77, 34), (130, 2, 2, 128, 0), (1200, 28, 4, 128, 128), (4, 1, 1, 1, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rotation_and_its_gradient(shape, layout, dtype):
    t, hq, hkv, d, rot = shape
    rng = np.random.default_rng(t * 131 + d)
    pos = rng.integers(0, 200000, t)
    q, k = make(rng, (t, hq, d), dtype), make(rng, (t, hkv, d), dtype)
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    f, factor = frequencies(rot, 10000.0, None) if rot else (np.zeros(0), 1.0)
    with rope.RopePlan(d=d, d_rot=rot, layout=layout, dtype=dtype) as plan:
        p = torch.from_numpy(pos).cuda()
        for sign, call in ((1, plan.rotate), (-1, plan.rotate_backward)):
            call(q, qo, k, ko, positions=p)
            for x, y in ((q, qo), (k, ko)):
                ref, mag = turn(f64(x), pos, rot, layout, f, factor, sign)
                near(y, ref, 16 * U * mag)
        # in place gives the same bits
        q2, k2 = q.clone(), k.clone()
        plan.rotate(q2, q2, k2, k2, positions=p)
        plan.rotate(q, qo, k, ko, positions=p)
        assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scalings_at_long_and_negative_positions(scaling, layout):
    pos = np.array([0, 1, 8191, 131071, 1048575, 2 ** 31 - 1, -5, -100000], np.int64)
    rng = np.random.default_rng(3)
    x = make(rng, (len(pos), 2, 128), "fp32")
    y = torch.empty_like(x)
    f, factor = frequencies(96, 500000.0, scaling)
    with rope.RopePlan(d=128, d_rot=96, layout=layout, base=500000.0, scaling=scaling, dtype="fp32") as plan:
        gf, ga = plan.frequencies()
        np.testing.assert_allclose(gf, f, rtol=1e-13)
        assert abs(ga - factor) < 1e-14
        plan.rotate(x, y, positions=torch.from_numpy(pos).cuda())
    # the 64-bit angle itself is rounded: |pos| * 2^-52 radians
    ref, mag = turn(f64(x), pos, 96, layout, f, factor)
    near(y, ref, (16 * U + np.abs(pos)[:, None, None] * 2.0 ** -51) * mag)


def norm_ref(x, w, eps):
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * w, r


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_rotation_and_its_gradient(shape, layout, dtype):
    t, hq, hkv, d, rot = shape
    rng = np.random.default_rng(t * 17 + d)
    pos = np.arange(t) + 1000
    f, factor = frequencies(rot, 10000.0, None) if rot else (np.zeros(0), 1.0)
    eps = 1e-5
    x = {n: make(rng, (t, h, d), dtype, 2.0) for n, h in (("q", hq), ("k", hkv))}
    dy = {n: make(rng, (t, h, d), dtype) for n, h in (("q", hq), ("k", hkv))}
    w = {n: make(rng, (d,), dtype) for n in "qk"}
    out = {n: torch.full_like(x[n], 7) for n in "qk"}
    dw = {n: torch.full((d,), 7.0, device="cuda") for n in "qk"}
    with rope.RopePlan(d=d, d_rot=rot, layout=layout, dtype=dtype) as plan:
        plan.norm_rotate(x["q"], out["q"], w["q"], x["k"], out["k"], w["k"], pos0=1000, eps=eps)
        for n in "qk":
            h, _ = norm_ref(f64(x[n]), f64(w[n]), eps)
            ref, mag = turn(h, pos, rot, layout, f, factor)
            near(out[n], ref, 64 * U * mag)
        plan.norm_rotate_backward(x["q"], dy["q"], out["q"], w["q"], dw["q"], x["k"], dy["k"], out["k"], w["k"], dw["k"],
                                  pos0=1000, eps=eps)
        again = {n: torch.empty_like(dw[n]) for n in "qk"}
        plan.norm_rotate_backward(x["q"], dy["q"], out["q"], w["q"], again["q"], x["k"], dy["k"], out["k"], w["k"],
                                  again["k"], pos0=1000, eps=eps)
    for n in "qk":
        xx, ww = f64(x[n]), f64(w[n])
        g, mag = turn(f64(dy[n]), pos, rot, layout, f, factor, -1)
        _, r = norm_ref(xx, ww, eps)
        h = xx * r
        ref = r * (g * ww - h * (g * ww * h).mean(-1, keepdims=True))
        size = r * (mag * np.abs(ww) + np.abs(h) * (mag * np.abs(ww * h)).mean(-1, keepdims=True))
        near(out[n], ref, 96 * U * size)
        rows = t * x[n].shape[1]
        near(dw[n], (g * h).sum((0, 1)), (rows + 128) * U * (mag * np.abs(h)).sum((0, 1)))
        assert torch.equal(dw[n], again[n])


def test_gradient_against_differences():
    t, h, d, rot, eps = 3, 2, 32, 24, 1e-6
    rng = np.random.default_rng(0)
    x, dy, w = make(rng, (t, h, d), "fp32"), make(rng, (t, h, d), "fp32"), make(rng, (d,), "fp32")
    pos = np.array([0, 77, 123456])
    f, factor = frequencies(rot, 10000.0, None)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    with rope.RopePlan(d=d, d_rot=rot, dtype="fp32") as plan:
        plan.norm_rotate_backward(x, dy, dx, w, dw, positions=torch.from_numpy(pos).cuda(), eps=eps)

    def loss(xx, ww):
        return float((turn(norm_ref(xx, ww, eps)[0], pos, rot, "half", f, factor)[0] * f64(dy)).sum())

    xx, ww, step = f64(x), f64(w), 1e-5
    for _ in range(8):
        a, b = rng.standard_normal(xx.shape), rng.standard_normal(ww.shape)
        diff = (loss(xx + step * a, ww) - loss(xx - step * a, ww)) / (2 * step)
        # differences: step^2 * third derivative and 1e-16 / step; the kernel: 96 * 2^-24 a term
        assert abs(diff - (f64(dx) * a).sum()) <= 1e-4 * np.abs(f64(dx) * a).sum()
        diff = (loss(xx, ww + step * b) - loss(xx, ww - step * b)) / (2 * step)
        assert abs(diff - (f64(dw) * b).sum()) <= 1e-4 * np.abs(f64(dw) * b).sum()


def test_packed_projection_into_cache_slots():
    """q, k, v as views of one projection; k and v land in scattered cache rows,
    negative and outside slots nowhere."""
    t, hq, hkv, d = 9, 4, 2, 128
    rng = np.random.default_rng(5)
    qkv = make(rng, (t, hq + 2 * hkv, d), "bf16")
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    slots = torch.tensor([5, 3, -1, 40, 0, 39, 7, 12, 41], device="cuda")
    pos = torch.arange(t, device="cuda") * 100
    kc = torch.full((40, hkv, d), 9.0, dtype=torch.bfloat16, device="cuda")
    vc, qo, ko = kc.clone(), torch.empty_like(q), torch.empty_like(k)
    w = make(rng, (d,), "bf16")
    with rope.RopePlan() as plan:
        plan.norm_rotate(q, qo, w, k, ko, w, positions=pos)
        q2 = torch.empty_like(q)
        plan.norm_rotate(q, q2, w, k, kc, w, v, vc, positions=pos, slots=slots)
    assert torch.equal(qo, q2)
    want_k, want_v = torch.full_like(kc, 9.0), torch.full_like(vc, 9.0)
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < 40:
            want_k[s], want_v[s] = ko[i], v[i]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


@pytest.mark.parametrize("t, hq, hkv, d, rot, layout, dtype", [
    (40001, 1, 1, 256, 256, "half", "bf16"), (20011, 1, 1, 256, 64, "interleaved", "fp32"),
    (9001, 5, 2, 128, 64, "half", "bf16"), (18007, 3, 2, 80, 48, "interleaved", "fp16"), (701, 1, 1, 77, 34, "half", "bf16")])
def test_many_rows_of_few_heads_into_slots(t, hq, hkv, d, rot, layout, dtype):
    """Several rows a lane, blocks of many tokens, rows of three tensors in one
    pass; every third slot is none."""
    rng = np.random.default_rng(t)
    q, k, v = make(rng, (t, hq, d), dtype), make(rng, (t, hkv, d), dtype), make(rng, (t, hkv, d), dtype)
    wq, wk = make(rng, (d,), dtype), make(rng, (d,), dtype)
    to = rng.permutation(t)
    to[::3] = rng.choice([-1, t, 2 ** 40], len(to[::3]))
    slots = torch.from_numpy(to).cuda()
    qo, ko, vo = torch.full_like(q, 7), torch.full_like(k, 7), torch.full_like(v, 7)
    f, factor = frequencies(rot, 10000.0, None)
    pos, eps = np.arange(t) + 31, 1e-6
    kept = (to >= 0) & (to < t)
    rest = np.setdiff1d(np.arange(t), to[kept])
    with rope.RopePlan(d=d, d_rot=rot, layout=layout, dtype=dtype) as plan:
        for norm in (True, False):
            if norm:
                plan.norm_rotate(q, qo, wq, k, ko, wk, v, vo, pos0=31, slots=slots, eps=eps)
            else:
                plan.rotate(q, qo, k, ko, v, vo, pos0=31, slots=slots)
            for x, w, y, rows in ((q, wq, qo, slice(None)), (k, wk, ko, kept)):
                h = norm_ref(f64(x)[rows], f64(w), eps)[0] if norm else f64(x)[rows]
                ref, mag = turn(h, pos[rows], rot, layout, f, factor)
                near(y if x is q else y[slots[torch.from_numpy(kept).cuda()]], ref, (64 if norm else 16) * U * mag)
            assert torch.equal(vo[slots[torch.from_numpy(kept).cuda()]], v[torch.from_numpy(kept).cuda()])
            assert (ko[torch.from_numpy(rest).cuda()] == 7).all() and (vo[torch.from_numpy(rest).cuda()] == 7).all()


def test_strides_and_streams():
    """Head-major tensors, an unaligned view, and a stream of the caller's."""
    rng = np.random.default_rng(6)
    base = make(rng, (4, 50, 64), "bf16")  # [heads, tokens, d]
    x = base.transpose(0, 1)
    odd = torch.zeros(50 * 4 * 65 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(50, 4, 65)[..., :64]
    odd.copy_(x)
    out, out2 = torch.empty_like(base).transpose(0, 1), torch.empty_like(odd)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with rope.RopePlan(d=64) as plan:
        plan.rotate(x, out, pos0=17, stream=st)
        plan.rotate(odd, out2, pos0=17, stream=st)
        st.synchronize()
        ref = torch.empty((50, 4, 64), dtype=torch.bfloat16, device="cuda")
        plan.rotate(x.contiguous(), ref, pos0=17)
    assert torch.equal(out, ref) and torch.equal(out2, ref)


def test_nothing_to_do():
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((64,), 3.0, device="cuda")
    with rope.RopePlan(d=64) as plan:
        plan.rotate(e, e)
        plan.norm_rotate_backward(e, e, e, w, dw)
    assert (dw == 0).all()


def test_non_finite_rows_stay_in_their_row():
    rng = np.random.default_rng(8)
    x = make(rng, (64, 2, 128), "bf16")
    y, z = torch.empty_like(x), torch.empty_like(x)
    bad = x.clone()
    bad[10, 1, 3], bad[20, 0, 100] = math.nan, math.inf
    w = make(rng, (128,), "bf16")
    with rope.RopePlan() as plan:
        plan.norm_rotate(x, y, w)
        plan.norm_rotate(bad, z, w)
    same = torch.ones(64, 2, dtype=torch.bool, device="cuda")
    same[10, 1] = same[20, 0] = False
    assert torch.equal(y[same], z[same]) and torch.isnan(z[10, 1]).all()


@pytest.mark.parametrize("cfg", [dict(d=0), dict(d=257), dict(d_rot=3), dict(d=64, d_rot=66), dict(base=1.0),
                                 dict(base=math.nan), dict(scaling=dict(kind="linear", factor=0.5)),
                                 dict(d_rot=2, scaling=dict(kind="ntk", factor=2.0)), dict(attn_factor=-1.0),
                                 dict(scaling=dict(kind="yarn", factor=2.0, beta_fast=1.0, beta_slow=2.0)),
                                 dict(scaling=dict(kind="llama3", factor=2.0, low_freq_factor=4.0))])
def test_refused_configurations(cfg):
    with pytest.raises(syn.SynError):
        rope.RopePlan(**cfg)


def test_refused_calls():
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda")
    with rope.RopePlan() as plan:
        for bad in (x.float(), x[..., :64], x[0], x.transpose(1, 2), x.cpu()):
            with pytest.raises(ValueError):
                plan.rotate(bad, bad)
        with pytest.raises(ValueError):
            plan.rotate(x, x[:3])
        with pytest.raises(ValueError):
            plan.rotate(x, x, positions=torch.zeros(4, dtype=torch.int32, device="cuda"))
        with pytest.raises(ValueError):
            plan.rotate(None, None)
        with pytest.raises(syn.SynError):
            plan.norm_rotate(x, x, None, eps=-1.0)
        L = rope.lib()
        assert L.syn_rope(None, None, None, None, None, 0, None, 0, 0, None) == syn.ERR_INVALID
        assert L.syn_rope(plan._h, None, None, None, None, 0, None, 0, -1, None) == syn.ERR_INVALID
        r = rope.Rows(0, 1, 1, 0, 1, 1, 2)
        assert L.syn_rope(plan._h, r, None, None, None, 0, None, 0, 4, None) == syn.ERR_INVALID


def test_gradient_without_weights_beside_one_with_them():
    """Calls that want no weight gradients run beside one of the same plan that does, on another stream."""
    rng = np.random.default_rng(12)
    t, h, d = 3000, 4, 128
    x, dy, w = make(rng, (t, h, d), "bf16"), make(rng, (t, h, d), "bf16"), make(rng, (d,), "bf16")
    x2, dy2 = make(rng, (t, h, d), "bf16", 3.0), make(rng, (t, h, d), "bf16", 3.0)
    dx, dx2, ref, ref2 = (torch.empty_like(x) for _ in range(4))
    dw, want = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with rope.RopePlan() as plan:
        plan.norm_rotate_backward(x, dy, ref, w, want)
        plan.norm_rotate_backward(x2, dy2, ref2, w, None)
        torch.cuda.synchronize()
        for _ in range(200):
            for _ in range(3):
                plan.norm_rotate_backward(x2, dy2, dx2, w, None, stream=b)
            plan.norm_rotate_backward(x, dy, dx, w, dw, stream=a)
            for _ in range(3):
                plan.norm_rotate_backward(x2, dy2, dx2, w, None, stream=b)
            torch.cuda.synchronize()
            assert torch.equal(dw, want) and torch.equal(dx, ref) and torch.equal(dx2, ref2)


def test_gradients_from_two_host_threads():
    """Two threads, each with a plan of its own, in calls that need different amounts of shared memory."""
    import threading

    rng = np.random.default_rng(14)
    failed = []

    def work(x, dy, w, want, gate):
        dx, st = torch.empty_like(x), torch.cuda.Stream()
        with rope.RopePlan() as plan:
            gate.wait()
            try:
                for _ in range(3000):
                    plan.norm_rotate_backward(x, dy, dx, w, None, stream=st)
                st.synchronize()
                assert torch.equal(dx, want)
            except BaseException as e:
                failed.append(e)

    threads, gate = [], threading.Barrier(2)
    for heads in (1, 64):  # a step spans many tokens' angles, or few
        x, dy, w = make(rng, (64 // heads, heads, 128), "bf16"), make(rng, (64 // heads, heads, 128), "bf16"), make(rng, (128,), "bf16")
        want = torch.empty_like(x)
        with rope.RopePlan() as plan:
            plan.norm_rotate_backward(x, dy, want, w, None)
        threads.append(threading.Thread(target=work, args=(x, dy, w, want, gate)))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[0]


def test_a_new_plan_on_another_stream():
    """The first call of a plan, on a stream that does not wait for the default one, while that one is busy."""
    rng = np.random.default_rng(15)
    x = make(rng, (64, 4, 256), "fp32")
    y, ref, busy = torch.empty_like(x), torch.empty_like(x), torch.zeros(1 << 26, device="cuda")
    with rope.RopePlan(d=256, dtype="fp32") as plan:
        plan.rotate(x, ref, pos0=1000)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(50):
        y.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            busy.add_(1)
        with rope.RopePlan(d=256, dtype="fp32") as plan:
            plan.rotate(x, y, pos0=1000, stream=st)
            st.synchronize()
            assert torch.equal(y, ref)


def test_overlapping_outputs_are_refused():
    rng = np.random.default_rng(19)
    x = make(rng, (4, 2, 64), "bf16")
    w, dw = make(rng, (64,), "bf16"), torch.empty(64, device="cuda")
    slots = torch.arange(4, device="cuda")
    base = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    bad = [base[:1].expand(4, 2, 64), base[:, :1].expand(4, 2, 64), base.view(-1).as_strided((4, 2, 64), (64, 32, 1))]
    with rope.RopePlan(d=64) as plan:
        for y in bad:
            with pytest.raises(syn.SynError):
                plan.rotate(x, y)
            with pytest.raises(syn.SynError):
                plan.norm_rotate(x, base, w, x, y, w, slots=slots)
            with pytest.raises(syn.SynError):
                plan.rotate_backward(x, y)
            with pytest.raises(syn.SynError):
                plan.norm_rotate_backward(x, x, y, w, dw)
        torch.cuda.synchronize()
        assert (base == 7).all()
        # broadcast inputs are read as they are, and one row may have any stride
        y, want = torch.empty_like(x), torch.empty_like(x)
        plan.rotate(x[:1].expand(4, 2, 64), y)
        plan.rotate(x[:1].expand(4, 2, 64).contiguous(), want)
        assert torch.equal(y, want)
        one = torch.empty_like(x[:1, :1])
        plan.rotate(x[:1, :1], one.as_strided((1, 1, 64), (0, 0, 1)))
        assert torch.equal(one, want[:1, :1])
