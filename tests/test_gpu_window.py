"""GPU parity of the windowed attention with sinks, its gradient and its
decoding step (include/syn_window.h) against a plain 64-bit implementation,
through the C ABI.

Tolerances, from the kernels' arithmetic, u the unit roundoff of the type
(2^-8 bf16, 2^-11 fp16), s = 2^-14 for everything in fp32 (scores, exp2, sums)
relative to the terms, and for fp16 half its subnormal spacing (2^-25) a term:

  O   the probabilities are rounded once: (u + s) sum p|v|
  dV  the same probabilities: (u + s) sum p|dO|
  dS  = p (dP - rowsum(dO * O)) with the stored O (its error times |dO|, and u|O|),
      rounded once: e = u|dS| + s p (|dP| + |rowsum|) + p sum |dO| (e_O + u|O|)
  dQ, dK  sums of scale * e |K| and scale * e |Q|

and each output is the rounding to its type of a value within these bounds.
lse: 2^-14 * max(1, |lse|).
"""
import math

import numpy as np
import pytest
import torch

from chunk_scheduled_communication_gb300 import syn, window

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8, 0.0), "fp16": (torch.float16, 2.0 ** -11, 2.0 ** -25)}
S = 2.0 ** -14


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    syn.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, ref, tol):
    """got is the rounding to its type of a value within tol of ref."""
    lo, hi = (f64(torch.from_numpy(ref + s * tol).to(got.dtype)) for s in (-1, 1))
    got = f64(got)
    assert ((lo <= got) & (got <= hi)).all(), float(np.maximum(lo - got, got - hi).max())


def make(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(TYPES[dtype][0]).cuda()


def mask(ql, kl, w, sinks):
    p = np.arange(kl - ql, kl)[:, None]
    j = np.arange(kl)[None]
    return (j <= p) & ((j > p - w) | (j < sinks) if w else True)


def reference(q, k, v, q_lens, k_lens, w, sinks, u, tiny, do=None, scale=None):
    """Outputs and error bounds in 64 bits, sequence by sequence, head by head."""
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    g, scale = hq // hkv, scale or 1 / math.sqrt(d)
    names = ["O", "eO"] + (["dQ", "eQ", "dK", "eK", "dV", "eV"] if do is not None else [])
    r = {n: np.zeros(q.shape if n[-1] in "OQ" else k.shape) for n in names}
    lse = np.full(q.shape[:2], -np.inf)
    q0 = k0 = 0
    for ql, kl in zip(q_lens, k_lens):
        see = mask(ql, kl, w, sinks)
        a, b = slice(q0, q0 + ql), slice(k0, k0 + kl)
        for h in range(hq):
            if ql == 0 or kl == 0:
                continue
            qq, kk, vv = q[a, h], k[b, h // g], v[b, h // g]
            s = np.where(see, qq @ kk.T * scale, -np.inf)
            top = s.max(-1, keepdims=True)
            e = np.exp(s - np.where(np.isfinite(top), top, 0))
            tot = e.sum(-1, keepdims=True)
            p = e / np.where(tot == 0, 1, tot)
            with np.errstate(divide="ignore"):
                lse[a, h] = np.where(tot == 0, -np.inf, np.log(tot) + top)[:, 0]
            r["O"][a, h] = p @ vv
            eo = (u + S) * (p @ np.abs(vv)) + tiny * (see @ np.abs(vv))
            r["eO"][a, h] = eo
            if do is None:
                continue
            dd = do[a, h]
            dp = dd @ vv.T
            delta = (dd * r["O"][a, h]).sum(-1, keepdims=True)
            ds = p * (dp - delta)
            e_delta = (np.abs(dd) * (eo + u * np.abs(r["O"][a, h]) + tiny)).sum(-1, keepdims=True)
            es = u * np.abs(ds) + S * p * (np.abs(dd) @ np.abs(vv).T + (np.abs(dd) * np.abs(r["O"][a, h])).sum(-1, keepdims=True)) \
                + p * e_delta + tiny * see
            r["dQ"][a, h] = scale * ds @ kk
            r["eQ"][a, h] = scale * es @ np.abs(kk)
            r["dK"][b, h // g] += scale * ds.T @ qq
            r["eK"][b, h // g] += scale * es.T @ np.abs(qq)
            r["dV"][b, h // g] += p.T @ dd
            r["eV"][b, h // g] += (u + S) * (p.T @ np.abs(dd)) + tiny * (see.T @ np.abs(dd))
        q0, k0 = q0 + ql, k0 + kl
    return r, lse


def near_lse(got, ref):
    got = f64(got)
    none = np.isneginf(ref)
    assert (np.isneginf(got) == none).all()
    assert (np.abs(got[~none] - ref[~none]) <= S * np.maximum(1, np.abs(ref[~none]))).all()


CASES = [  # q_lens, k_lens, hq, hkv, d, window, sinks
    ([1], [1], 1, 1, 128, 0, 0),
    ([128], [128], 2, 1, 128, 0, 0),
    ([129], [129], 2, 2, 64, 64, 0),
    ([300], [300], 4, 1, 128, 100, 4),
    ([5, 0, 260, 1], [5, 0, 260, 1], 4, 2, 64, 33, 2),
    ([257], [257], 3, 1, 128, 128, 130),
    ([64, 200, 31], [500, 200, 64], 2, 1, 128, 150, 16),
    ([200, 7, 40], [130, 0, 1], 2, 1, 64, 20, 4),       # rows without a key
    ([700], [700], 1, 1, 64, 1, 0),                      # only the key itself
    ([700], [700], 2, 1, 128, 1, 1),
    ([1], [1000], 8, 2, 128, 300, 4),                    # one new token
    ([513], [513], 6, 2, 64, 0, 0),
    ([384], [384], 2, 2, 128, 1000, 64),                 # a window longer than the keys
    ([90, 90, 90], [90, 90, 90], 10, 2, 128, 32, 33),
]


def setup(case, dtype, seed=0):
    q_lens, k_lens, hq, hkv, d, w, sinks = case
    rng = np.random.default_rng(seed + sum(q_lens) * 7 + d + w)
    q, k, v = make(rng, (sum(q_lens), hq, d), dtype), make(rng, (sum(k_lens), hkv, d), dtype), make(rng, (sum(k_lens), hkv, d), dtype)
    do = make(rng, q.shape, dtype)
    return q, k, v, do


def plan_of(case, dtype, backward=True, **more):
    q_lens, k_lens, hq, hkv, d, w, sinks = case
    return window.WindowPlan(q_lens, k_lens, H_q=hq, H_kv=hkv, d=d, window=w, sinks=sinks, dtype=dtype, backward=backward, **more)


def run(plan, q, k, v, do=None, stream=None):
    out, lse = torch.full_like(q, 7), torch.full(q.shape[:2], 7.0, device="cuda")
    plan.forward(q, k, v, out, lse=lse, stream=stream)
    if do is None:
        plan.check(stream)
        return out, lse
    g = [torch.full_like(x, 7) for x in (q, k, v)]
    plan.backward(do, q, k, v, out, lse, *g, stream=stream)
    plan.check(stream)
    return (out, lse, *g)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_gradient(case, dtype):
    _, u, tiny = TYPES[dtype]
    q, k, v, do = setup(case, dtype)
    r, lse_ref = reference(f64(q), f64(k), f64(v), case[0], case[1], case[5], case[6], u, tiny, f64(do))
    with plan_of(case, dtype) as plan:
        out, lse, dq, dk, dv = run(plan, q, k, v, do)
        again = run(plan, q, k, v, do)
    near(out, r["O"], r["eO"])
    near_lse(lse, lse_ref)
    near(dq, r["dQ"], r["eQ"])
    near(dk, r["dK"], r["eK"])
    near(dv, r["dV"], r["eV"])
    for a, b in zip((out, lse, dq, dk, dv), again):
        assert torch.equal(a, b)


def test_many_items_per_cta():
    """More items than a CTA keeps in shared memory, and sequences of every residue."""
    lens = [1 + 37 * i % 150 for i in range(400)]
    case = (lens, lens, 16, 16, 64, 40, 3)
    q, k, v, do = setup(case, "bf16")
    _, u, tiny = TYPES["bf16"]
    r, lse_ref = reference(f64(q), f64(k), f64(v), lens, lens, 40, 3, u, tiny, f64(do))
    with plan_of(case, "bf16") as plan:
        assert plan.info()["n_items"] > 48 * 100
        out, lse, dq, dk, dv = run(plan, q, k, v, do)
    near(out, r["O"], r["eO"])
    near_lse(lse, lse_ref)
    for got, n in ((dq, "Q"), (dk, "K"), (dv, "V")):
        near(got, r["d" + n], r["e" + n])


def test_large_scores_and_scale():
    """Scores of hundreds: the reference maximum moves by more than its slack."""
    case = ([260], [260], 2, 1, 128, 90, 4)
    q, k, v, do = setup(case, "bf16")
    k = (k.float() * torch.linspace(0.1, 6, 260, device="cuda")[:, None, None]).to(k.dtype)
    _, u, tiny = TYPES["bf16"]
    r, lse_ref = reference(f64(q), f64(k), f64(v), [260], [260], 90, 4, u, tiny, scale=0.5)
    # a score's fp32 error is relative to the score: up to ~500 here
    with plan_of(case, "bf16", scale=0.5) as plan:
        out, lse = run(plan, q, k, v)
    near(out, r["O"], r["eO"] * 2)
    near_lse(lse, lse_ref)


def test_gradient_against_differences():
    case = ([70, 33], [70, 40], 4, 2, 64, 20, 3)
    q, k, v, do = setup(case, "fp16")
    _, u, tiny = TYPES["fp16"]
    args = (case[0], case[1], case[5], case[6], u, tiny)
    qq, kk, vv, dd = f64(q), f64(k), f64(v), f64(do)
    r, _ = reference(qq, kk, vv, *args, dd)
    with plan_of(case, "fp16") as plan:
        grads = [f64(x) for x in run(plan, q, k, v, do)[2:]]
    rng, step = np.random.default_rng(1), 1e-4
    for x, g, n in ((0, grads[0], "Q"), (1, grads[1], "K"), (2, grads[2], "V")):
        for _ in range(3):
            a = rng.standard_normal(g.shape)
            at = [qq, kk, vv]
            hi, lo = list(at), list(at)
            hi[x], lo[x] = at[x] + step * a, at[x] - step * a
            diff = sum(s * (reference(*y, *args)[0]["O"] * dd).sum() for s, y in ((1, hi), (-1, lo))) / (2 * step)
            # the kernel's bound and its rounding, and the differences' step^2
            tol = ((r["e" + n] + (u * np.abs(g)) + tiny) * np.abs(a)).sum() + 1e-5 * np.abs(g * a).sum()
            assert abs(diff - (g * a).sum()) <= tol


@pytest.mark.parametrize("d", [64, 128])
def test_other_sequences_do_not_reach_a_sequence(d):
    """Not finite anywhere in the neighbours: the same bits in the middle."""
    lens, klens = [70, 201, 90], [70, 230, 90]
    case = (lens, klens, 2, 1, d, 50, 5)
    q, k, v, do = setup(case, "bf16")
    with plan_of(case, "bf16") as plan:
        want = run(plan, q, k, v, do)
        for bad in (math.nan, math.inf):
            x = [t.clone() for t in (q, k, v, do)]
            for t, l in zip(x, (lens, klens, klens, lens)):
                t[:l[0]] = bad
                t[l[0] + l[1]:] = bad
            got = run(plan, *x)
            for a, b, l in zip(got, want, (lens, lens, lens, klens, klens)):
                assert torch.equal(a[l[0]:l[0] + l[1]], b[l[0]:l[0] + l[1]])


def test_non_finite_keys_that_no_row_sees():
    """Keys older than every window, and a not finite query row, stay where they are."""
    case = ([40], [600], 2, 1, 128, 64, 4)
    q, k, v, do = setup(case, "bf16")
    with plan_of(case, "bf16") as plan:
        want = run(plan, q, k, v, do)
        k2, v2 = k.clone(), v.clone()
        k2[4:480], v2[4:480] = math.nan, math.inf
        got = run(plan, q, k2, v2, do)
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
        q2 = q.clone()
        q2[7, 1] = math.nan
        out, lse = run(plan, q2, k, v)
    assert torch.isnan(out[7, 1]).all() and torch.isnan(lse[7, 1])
    rest = torch.ones(40, 2, dtype=torch.bool, device="cuda")
    rest[7, 1] = False
    assert torch.equal(out[rest], want[0][rest])


def test_strides_and_stream():
    """Views of one packed projection, head-major tensors, and a stream of the caller's."""
    case = ([300, 21], [300, 21], 4, 2, 64, 100, 4)
    q, k, v, do = setup(case, "bf16")
    t = 321
    qkv = torch.cat([q, k, v], 1)
    views = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    major = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, do)]
    st = torch.cuda.Stream()
    with plan_of(case, "bf16") as plan:
        want = run(plan, q, k, v, do)
        got = run(plan, *views, do)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got = run(plan, *major)
            out = torch.empty((4, t, 64), dtype=q.dtype, device="cuda").transpose(0, 1)
            lse = torch.empty((t, 4), device="cuda")
            plan.forward(*major[:3], out, lse=lse)
            g = [torch.empty_like(x) for x in (qkv, qkv)]
            plan.backward(do, *views, out, lse, g[0][:, :4], g[0][:, 4:6], g[0][:, 6:])
            plan.check()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(out, want[0])
        assert torch.equal(g[0], torch.cat(want[2:], 1))


def test_without_rows_or_keys():
    z = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.randn(5, 2, 64, device="cuda").bfloat16()
    for ql, kl in (([], []), ([0], [0]), ([5], [0]), ([0], [5])):
        with window.WindowPlan(ql, kl, H_q=2, H_kv=2, d=64, window=3, backward=True) as plan:
            a, b = (q if sum(ql) else z), (q if sum(kl) else z)
            out, lse, dq, dk, dv = run(plan, a, b, b, a)
            assert not out.any() and torch.isneginf(lse).all() and not dq.any() and not dk.any() and not dv.any()


@pytest.mark.parametrize("kw", [dict(d=96), dict(H_q=3, H_kv=2), dict(H_q=0), dict(window=-1), dict(sinks=-1),
                                dict(dtype="fp32"), dict(scale=-1.0), dict(scale=math.inf)])
def test_refused_plans(kw):
    with pytest.raises(syn.SynError):
        window.WindowPlan([4], **kw)
    with pytest.raises(syn.SynError):
        window.DecodePlan(max_seqs=2, **kw)


def test_refused_calls():
    with pytest.raises(syn.SynError):
        window.WindowPlan([-1])
    with pytest.raises(syn.SynError):
        window.WindowPlan([1 << 29])
    with pytest.raises(ValueError):
        window.WindowPlan([1, 2], [1])
    with pytest.raises(syn.SynError):
        window.DecodePlan(max_seqs=0)
    with pytest.raises(syn.SynError):
        window.DecodePlan(page_size=0)
    x = torch.zeros((8, 1, 128), dtype=torch.bfloat16, device="cuda")
    with window.WindowPlan([8]) as plan:
        for bad in (x.half(), x[:7], x.cpu(), x[..., :64]):
            with pytest.raises(ValueError):
                plan.forward(bad, x, x, x)
        with pytest.raises(ValueError):
            plan.forward(x, x, x, x, lse=torch.zeros(8, 1, dtype=torch.float64, device="cuda"))
        lse = torch.zeros(8, 1, device="cuda")
        with pytest.raises(syn.SynError):  # made without backward
            plan.backward(x, x, x, x, x, lse, x, x, x)
        pad = torch.zeros(8 * 132, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(syn.SynError):  # a stride that is not a multiple of 8
            plan.forward(pad.view(8, 1, 132)[..., :128], x, x, x)
        with pytest.raises(syn.SynError):  # not 16-byte aligned
            plan.forward(pad[1:1025].view(8, 1, 128), x, x, x)
        with pytest.raises(syn.SynError):  # a broadcast row
            plan.forward(x[:1].expand(8, 1, 128), x, x, x)
    L = window.lib()
    assert L.syn_window_attention(None, None, None, None, None, None, None) == syn.ERR_INVALID
    assert L.syn_window_decode(None, None, None, None, None, 0, 0, None, 1, None, None, None) == syn.ERR_INVALID


# ------------------------------------------------------------------ decoding
def paged(rng, lens, page, hkv, d, dtype, spare=5):
    per = max((n + page - 1) // page for n in lens) or 1
    pages = sum((n + page - 1) // page for n in lens) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), per), 2 ** 31 - 1, np.int32)  # entries that are never read
    kc, vc = make(rng, (pages, page, hkv, d), dtype), make(rng, (pages, page, hkv, d), dtype)
    kc[torch.from_numpy(order[len(order) - spare:]).cuda()] = math.nan
    vc[torch.from_numpy(order[len(order) - spare:]).cuda()] = math.nan
    at = 0
    for i, n in enumerate(lens):
        m = (n + page - 1) // page
        table[i, :m] = order[at:at + m]
        at += m
        if n % page:  # the last page's unused rows
            kc[int(table[i, m - 1]), n % page:] = math.nan
            vc[int(table[i, m - 1]), n % page:] = math.inf
    return kc, vc, torch.from_numpy(table).cuda()


def check_decode(q, kc, vc, table, lens, w, sinks, out, lse, u, tiny):
    page = kc.shape[1]
    t = table.cpu().numpy()
    for i, n in enumerate(lens):
        j = np.arange(n)
        seen = j[(j > n - 1 - w) | (j < sinks)] if w else j
        rows = t[i, seen // page], seen % page
        k, v = f64(kc)[rows], f64(vc)[rows]
        r, ls = reference(f64(q[i:i + 1]), k, v, [1], [len(seen)], 0, 0, u, tiny)
        near(out[i:i + 1], r["O"], r["eO"])
        near_lse(lse[i:i + 1], ls)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", [  # lens, hq, hkv, d, window, sinks, page
    ([1], 1, 1, 128, 0, 0, 16), ([0, 3, 64, 65], 8, 2, 64, 0, 0, 16), ([500, 20, 1000, 999], 4, 1, 128, 100, 4, 64),
    ([2000], 7, 1, 128, 600, 70, 32), ([300, 310], 20, 1, 64, 64, 1, 1), ([700, 1], 40, 2, 128, 1, 0, 7),
    ([1500] * 3, 16, 16, 64, 0, 0, 100)])
def test_decode(case, dtype):
    lens, hq, hkv, d, w, sinks, page = case
    _, u, tiny = TYPES[dtype]
    rng = np.random.default_rng(sum(lens) + d)
    kc, vc, table = paged(rng, lens, page, hkv, d, dtype)
    for i, n in enumerate(lens):  # pages without a visible key are not read
        for e in range(table.shape[1]):
            if w and e * page >= sinks and (e + 1) * page <= n - w:
                kc[int(table[i, e])], vc[int(table[i, e])] = math.nan, math.nan
    q = make(rng, (len(lens), hq, d), dtype)
    out, lse = torch.full_like(q, 7), torch.empty((len(lens), hq), device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    with window.DecodePlan(max_seqs=len(lens) + 2, H_q=hq, H_kv=hkv, d=d, window=w, sinks=sinks, page_size=page, dtype=dtype) as plan:
        plan.run(q, kc, vc, sl, out, lse=lse, page_table=table)
        plan.check()
        check_decode(q, kc, vc, table, lens, w, sinks, out, lse, u, tiny)
        for _ in range(3):  # the same bits, whatever range arrives last
            out2 = torch.empty_like(out)
            plan.run(q, kc, vc, sl, out2, page_table=table)
            assert torch.equal(out, out2)


def test_decode_equals_forward_on_a_contiguous_cache():
    """The last row of a prompt, through the forward and through the decoding step."""
    rng = np.random.default_rng(2)
    b, s, hq, hkv, d, w, sinks = 2, 400, 8, 2, 128, 150, 4
    k, v = make(rng, (b, 512, hkv, d), "bf16"), make(rng, (b, 512, hkv, d), "bf16")
    q = make(rng, (b * s, hq, d), "bf16")
    u = TYPES["bf16"][1]
    with window.WindowPlan([s] * b, H_q=hq, H_kv=hkv, window=w, sinks=sinks) as plan:
        out, _ = run(plan, q, k[:, :s].reshape(-1, hkv, d).contiguous(), v[:, :s].reshape(-1, hkv, d).contiguous())
    one = torch.empty((b, hq, d), dtype=q.dtype, device="cuda")
    with window.DecodePlan(max_seqs=b, H_q=hq, H_kv=hkv, window=w, sinks=sinks, page_size=512) as plan:
        plan.run(q.view(b, s, hq, d)[:, -1], k, v, torch.full((b,), s, dtype=torch.int32, device="cuda"), one)
        plan.check()
    a, c = f64(one), f64(out.view(b, s, hq, d)[:, -1])
    # both within (2u + s) of sum p|v| <= max|v|
    assert (np.abs(a - c) <= 2 * (2 * u + S) * f64(v).max()).all()


def test_decode_reports_what_is_out_of_range():
    rng = np.random.default_rng(3)
    k, v = make(rng, (4, 16, 1, 64), "bf16"), make(rng, (4, 16, 1, 64), "bf16")
    q = make(rng, (3, 1, 64), "bf16")
    out, ok = torch.empty_like(q), torch.empty_like(q)
    lens = torch.tensor([16, 40, -3], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 9], [1, 2], [3, 3]], dtype=torch.int32, device="cuda")
    with window.DecodePlan(max_seqs=3, d=64, page_size=16) as plan:
        plan.run(q, k, v, lens, out, page_table=table)  # 40 > 32 keys, -3
        assert plan.sync() == syn.ERR_BOUNDS
        assert plan.sync() == syn.OK
        assert not out[2].any()
        plan.run(q, k, v, torch.tensor([16, 32, 0], dtype=torch.int32, device="cuda"), ok, page_table=table)
        plan.check()
        assert torch.equal(out, ok)
        plan.run(q, k, v, torch.tensor([17, 0, 0], dtype=torch.int32, device="cuda"), ok, page_table=table)  # page 9
        assert plan.sync() == syn.ERR_BOUNDS
        assert torch.equal(ok[0], out[0])
        for bad in (dict(seq_lens=lens.long()), dict(seq_lens=lens[:2]), dict(page_table=table.long()), dict(page_table=table[:2])):
            with pytest.raises(ValueError):
                plan.run(q, k, v, bad.get("seq_lens", lens), out, page_table=bad.get("page_table", table))
        with pytest.raises(syn.SynError):  # more sequences than the plan's
            plan.run(torch.cat([q, q]), k, v, torch.cat([lens, lens]), torch.cat([q, q]), page_table=torch.cat([table, table]))
        with pytest.raises(ValueError):
            plan.run(q, k[:, :8], v, lens, out, page_table=table)


@pytest.mark.parametrize("w, sinks", [(0, 0), (64, 4)])
@pytest.mark.parametrize("n", [33, 2**30 + 40, 2**31 - 1])
def test_decode_lengths_past_the_table(w, sinks, n):
    # the keys that the table names and the window shows remain, however long the sequence claims to be
    rng = np.random.default_rng(11)
    k, v, q = make(rng, (4, 16, 1, 64), "bf16"), make(rng, (4, 16, 1, 64), "bf16"), make(rng, (2, 1, 64), "bf16")
    table = torch.tensor([[2, 1], [0, 3]], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((2, 1), dtype=torch.float32, device="cuda")
    with window.DecodePlan(max_seqs=2, d=64, window=w, sinks=sinks, page_size=16) as plan:
        plan.run(q, k, v, torch.tensor([n, 5], dtype=torch.int32, device="cuda"), out, page_table=table, lse=lse)
        assert plan.sync() == syn.ERR_BOUNDS
        assert plan.sync() == syn.OK
    first = max(n - min(w or 2**30, 2**30), 0)
    seen = [j for j in range(32) if j >= first or j < sinks]
    if not seen:
        assert not out[0].any() and lse[0].item() == -np.inf
        return
    keys, vals = (f64(x)[[2, 1]].reshape(32, 64)[seen] for x in (k, v))
    scores = keys @ f64(q)[0, 0] / 8
    weights = np.exp(scores - scores.max())
    want = weights @ vals / weights.sum()
    u = TYPES["bf16"][1]
    assert (np.abs(f64(out)[0, 0] - want) <= (2 * u + S) * np.abs(vals).max()).all()


def test_decode_reports_pages_below_zero():
    rng = np.random.default_rng(12)
    k, v, q = make(rng, (2, 16, 1, 64), "bf16"), make(rng, (2, 16, 1, 64), "bf16"), make(rng, (1, 1, 64), "bf16")
    out, ok = torch.empty_like(q), torch.empty_like(q)
    with window.DecodePlan(max_seqs=1, d=64, page_size=16) as plan:
        for page in (-1, -2, -2**31):
            table = torch.tensor([[1, page]], dtype=torch.int32, device="cuda")
            plan.run(q, k, v, torch.tensor([20], dtype=torch.int32, device="cuda"), out, page_table=table)
            assert plan.sync() == syn.ERR_BOUNDS
            plan.run(q, k, v, torch.tensor([16], dtype=torch.int32, device="cuda"), ok, page_table=table)
            plan.check()
            assert torch.equal(out, ok)


def test_dependent_calls_back_to_back_and_in_a_graph():
    """Each call reads what the one before wrote and overwrites what it read;
    the same bits with a pause after each call, without, and replayed."""
    from chunk_scheduled_communication_gb300 import rope

    rng = np.random.default_rng(21)
    lens, hq, hkv, d, page = [70, 1, 333], 4, 2, 64, 16
    n = sum(lens)
    x0 = [make(rng, (n, h, d), "bf16") for h in (hq, hkv, hkv)]
    do, w = make(rng, (n, hq, d), "bf16"), make(rng, (d,), "bf16")
    x = [t.clone() for t in x0]
    out, lse = torch.empty_like(x[0]), torch.empty((n, hq), device="cuda")
    g = [torch.empty_like(t) for t in x]
    k_rows, v_rows = (torch.zeros((n + page, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.arange(n, device="cuda")
    pages = -(-n // page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    length, one = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.empty((1, hq, d), dtype=torch.bfloat16, device="cuda")
    with rope.RopePlan(d=d) as turn, window.WindowPlan(lens, H_q=hq, H_kv=hkv, d=d, window=50, sinks=2, backward=True) as plan, \
            window.DecodePlan(max_seqs=1, H_q=hq, H_kv=hkv, d=d, window=50, sinks=2, page_size=page) as step:
        def calls(pause):
            for i in range(3):
                turn.norm_rotate(x[0], x[0], w, x[1], x[1], w)  # in place
                pause()
                plan.forward(*x, out, lse=lse)
                pause()
                plan.backward(do, *x, out, lse, *g)
                pause()
                turn.rotate(g[0], x[0], g[1], k_rows, g[2], v_rows, slots=slots)
                pause()
                step.run(x[0][-1:], k_rows[:pages * page].view(pages, page, hkv, d), v_rows[:pages * page].view(pages, page, hkv, d),
                         length, one, page_table=table)
                pause()
                turn.rotate(k_rows[:n], x[1], v_rows[:n], x[2])
                pause()

        def start():
            for a, b in zip(x, x0):
                a.copy_(b)

        def result():
            torch.cuda.synchronize()
            got = [t.clone() for t in (*x, out, lse, *g, k_rows, v_rows, one)]
            return got

        start()
        calls(torch.cuda.synchronize)
        want = result()
        assert all(t.isfinite().all() for t in want)
        for _ in range(20):
            start()
            calls(lambda: None)
            assert all(torch.equal(a, b) for a, b in zip(result(), want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            start()
            calls(lambda: None)
        for _ in range(3):
            for t in x:
                t.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(result(), want))
        plan.check()
        step.check()


def test_an_error_after_a_cleared_one_is_reported():
    rng = np.random.default_rng(16)
    k, v, q = make(rng, (2, 16, 1, 64), "bf16"), make(rng, (2, 16, 1, 64), "bf16"), make(rng, (1, 1, 64), "bf16")
    out, table = torch.empty_like(q), torch.tensor([[1, 7]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with window.DecodePlan(max_seqs=1, d=64, page_size=16) as plan:
        for _ in range(200):
            plan.run(q, k, v, lens, out, page_table=table, stream=st)  # page 7 of 2
            assert plan.sync(st) == syn.ERR_BOUNDS
        assert plan.sync(st) == syn.OK


def test_decode_waits_that_run_out(monkeypatch):
    """A limit that no wait is sure to meet: the call ends, says what happened, and the next one is right."""
    rng = np.random.default_rng(17)
    b, page, d = 64, 64, 128
    pages = b * 32
    k, v = (torch.randn((pages, page, 4, d), device="cuda").bfloat16() for _ in range(2))
    q, out, ref = make(rng, (b, 8, d), "bf16"), *(torch.empty((b, 8, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32).reshape(b, 32)).cuda()
    lens = torch.full((b,), 32 * page, dtype=torch.int32, device="cuda")
    with window.DecodePlan(max_seqs=b, H_q=8, H_kv=4, window=1024, sinks=4, page_size=page) as plan:
        plan.run(q, k, v, lens, ref, page_table=table)
        plan.check()
        for _ in range(5):
            monkeypatch.setenv("SYN_TIMEOUT_NS", "1")
            plan.run(q, k, v, lens, out, page_table=table)
            status = plan.sync()
            assert status in (syn.OK, syn.ERR_TIMEOUT)
            if status == syn.ERR_TIMEOUT:
                assert b"time limit" in syn.lib().syn_last_error()
            monkeypatch.delenv("SYN_TIMEOUT_NS")
            plan.run(q, k, v, lens, out, page_table=table)
            plan.check()
            assert torch.equal(out, ref)


def test_decode_strides_of_single_entries():
    """A stride of an axis with one entry is never used, whatever it is."""
    rng = np.random.default_rng(18)
    k, v, q = make(rng, (1, 64, 1, 64), "bf16"), make(rng, (1, 64, 1, 64), "bf16"), make(rng, (1, 1, 64), "bf16")
    k1, v1 = make(rng, (3, 1, 1, 64), "bf16"), make(rng, (3, 1, 1, 64), "bf16")

    def odd(t, axes):
        return t.as_strided(t.shape, [67 if i in axes else s for i, s in enumerate(t.stride())])

    for kc, vc, n, axes in ((k, v, 50, (0, 2)), (k1, v1, 1, (1, 2))):
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        want, got = torch.empty_like(q), torch.full_like(q, 7)
        with window.DecodePlan(max_seqs=1, d=64, page_size=kc.shape[1]) as plan:
            plan.run(q, kc, vc, lens, want)
            plan.run(odd(q, (0, 1)), odd(kc, axes), odd(vc, axes), lens, odd(got, (0, 1)))
            plan.check()
            assert torch.equal(got, want)
            two = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
            with pytest.raises(syn.SynError):  # used: refused as before
                plan.run(q, torch.zeros(67 * 64 + 64, dtype=torch.bfloat16, device="cuda").as_strided((2, *kc.shape[1:]), (67, 64, 64, 1)),
                         two.view(2, 1, 1, 64).expand(2, *kc.shape[1:]), lens, want)


def test_decode_refuses_a_broadcast_output():
    x = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    q, lens = x[:, 0], torch.tensor([3] * 4, dtype=torch.int32, device="cuda")
    with window.DecodePlan(max_seqs=4, H_q=2, H_kv=2, d=64, page_size=16) as plan:
        for bad in (q[:1].expand(4, 2, 64), q[:, :1].expand(4, 2, 64)):
            with pytest.raises(syn.SynError):
                plan.run(q, x, x, lens, bad)
        plan.run(q[:1].expand(4, 2, 64), x, x, lens, torch.empty_like(q))  # (a broadcast query is read as it is)
        plan.check()


def test_decode_with_an_empty_table_or_cache():
    """A table without pages names no key; it is not a missing table."""
    rng = np.random.default_rng(20)
    k, v, q = make(rng, (3, 16, 1, 64), "bf16"), make(rng, (3, 16, 1, 64), "bf16"), make(rng, (2, 1, 64), "bf16")
    out, lse = torch.full_like(q, 7), torch.full((2, 1), 7.0, device="cuda")
    table = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    with window.DecodePlan(max_seqs=2, d=64, page_size=16) as plan:
        for kc, vc in ((k, v), (k[:0], v[:0]), (torch.empty_like(k[:0]), torch.empty_like(v[:0]))):
            for n, status in (([5, 0], syn.ERR_BOUNDS), ([0, 0], syn.OK)):
                out.fill_(7), lse.fill_(7)
                plan.run(q, kc, vc, torch.tensor(n, dtype=torch.int32, device="cuda"), out, lse=lse, page_table=table)
                assert plan.sync() == status
                assert not out.any() and torch.isneginf(lse).all()


def test_overlapping_outputs_are_refused():
    x = torch.zeros((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((6, 2), device="cuda")
    bad = [x.view(-1).as_strided((6, 2, 64), s) for s in ((8, 64, 1), (128, 8, 1), (32, 384, 1))]
    c = torch.zeros((6, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([3] * 6, dtype=torch.int32, device="cuda")
    with window.WindowPlan([6], H_q=2, H_kv=2, d=64, backward=True) as plan, \
            window.DecodePlan(max_seqs=6, H_q=2, H_kv=2, d=64, page_size=16) as step:
        for y in bad:
            with pytest.raises(syn.SynError):
                plan.forward(x, x, x, y)
            for i in range(3):
                g = [torch.zeros_like(x) for _ in range(3)]
                g[i] = y
                with pytest.raises(syn.SynError):
                    plan.backward(x, x, x, x, x, lse, *g)
            with pytest.raises(syn.SynError):
                step.run(x, c, c, lens, y)


def test_a_sequence_of_thousands_of_rows():
    """Many blocks a row, sums in parts, a window and sinks far apart."""
    case = ([2503], [2700], 2, 1, 128, 900, 20)
    q, k, v, do = setup(case, "bf16")
    _, u, tiny = TYPES["bf16"]
    r, lse_ref = reference(f64(q), f64(k), f64(v), case[0], case[1], case[5], case[6], u, tiny, f64(do))
    with plan_of(case, "bf16") as plan:
        assert plan.info()["n_parts"] > 0
        out, lse, dq, dk, dv = run(plan, q, k, v, do)
    near(out, r["O"], r["eO"])
    near_lse(lse, lse_ref)
    near(dq, r["dQ"], r["eQ"])
    near(dk, r["dK"], r["eK"])
    near(dv, r["dV"], r["eV"])


def test_waits_that_run_out():
    """A limit that no wait is sure to meet: the calls end, and the next plan's are right."""
    case = ([1500, 3], [1500, 3], 4, 2, 128, 0, 0)
    q, k, v, do = setup(case, "bf16")
    with plan_of(case, "bf16") as plan, plan_of(case, "bf16", timeout_ns=1) as short:
        want = run(plan, q, k, v, do)
        got = [torch.empty_like(t) for t in want]
        for _ in range(3):
            short.forward(q, k, v, got[0], lse=got[1])
            status = short.sync()
            assert status in (syn.OK, syn.ERR_TIMEOUT)
            short.backward(do, q, k, v, want[0], want[1], *got[2:])
            assert short.sync() in (syn.OK, syn.ERR_TIMEOUT)
            assert all(torch.equal(a, b) for a, b in zip(run(plan, q, k, v, do), want))
