"""GPU parity of the layer norm and its gradient (include/syn_norm.h) against plain
64-bit implementations, through the C ABI.

Tolerances, from the kernels' arithmetic (U = 2^-24, half a step of fp32; outputs are
compared with the roundings of the tolerance's two ends).  A sum over a row runs over
at most 32 elements a lane and 10 levels of lanes and warps, so it is within 64 U of
the sum of magnitudes: the mean within em = 64 U mean|x|, so a deviation within em and
its rounding, the variance's root within 72 U and 2 em / sigma of itself (its sum, the
root within 2 ulp, the deviations' error), h = (x - m) / sigma within
eh = em/sigma (1 + 2 |h|) + 76 U |h|.  The output adds two roundings.  The gradient's means are
sums of the same kind, with h's error in one of them.  A weight gradient sums n rows
in chains: within (n + 128) U of the sum of magnitudes, and h's errors.
"""
import numpy as np
import pytest
import torch

from chunk_scheduled_communication_gb300 import norm, syn

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


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


def stats(x, eps):
    m = x.mean(-1, keepdims=True)
    inv = 1 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    h = (x - m) * inv
    em = 64 * U * np.abs(x).mean(-1, keepdims=True)
    return inv, h, em, em * inv * (1 + 2 * np.abs(h)) + 76 * U * np.abs(h)


def forward(x, w, b, eps):
    inv, h, em, eh = stats(x, eps)
    y = h * w + b
    return y, eh * np.abs(w) + 2 * U * (np.abs(h * w) + np.abs(y))


def backward(x, dy, w, eps):
    inv, h, em, eh = stats(x, eps)
    g = dy * w
    mg, mh = g.mean(-1, keepdims=True), (g * h).mean(-1, keepdims=True)
    dx = inv * (g - mg - h * mh)
    mean = lambda v: np.abs(v).mean(-1, keepdims=True)
    tol = inv * (8 * U * np.abs(g) + 72 * U * mean(g) + np.abs(h) * (80 * U * mean(g * h) + mean(np.abs(g) * eh))
                 + eh * np.abs(mh))
    tol += (76 * U + 2 * em * inv) * inv * (np.abs(g) + np.abs(mg) + np.abs(h * mh))
    n = (len(x) + 128) * U
    return dx, tol, ((dy * h).sum(0), (n * np.abs(dy * h) + np.abs(dy) * eh).sum(0)), (dy.sum(0), n * np.abs(dy).sum(0))


def make(rng, shape, dtype, scale=1.0, shift=0.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale + shift).astype(np.float32)).to(TYPES[dtype]).cuda()


def check(x, dy, w, b, eps=1e-5, plan=None, inplace=False):
    """Forward and gradient of x [n, d] (w, b: tensors or None) against 64 bits."""
    n, d = x.shape
    dtype = next(k for k, t in TYPES.items() if t is x.dtype)
    plan = plan or norm.NormPlan(d=d, dtype=dtype)
    x0, g0 = f64(x), f64(dy)
    w0, b0 = np.ones(d) if w is None else f64(w), np.zeros(d) if b is None else f64(b)
    keep = x.clone()
    y = x if inplace else torch.full_like(x, 7)
    plan.forward(x, y, w, b, eps=eps)
    near(y, *forward(x0, w0, b0, eps))
    x = keep
    dw, db = (torch.full((d,), 7.0, device="cuda") for _ in range(2))
    dx = dy if inplace else torch.full_like(x, 7)
    plan.backward(x, dy, dx, w, dw, db, eps=eps)
    ref, tol, (rw, tw), (rb, tb) = backward(x0, g0, w0, eps)
    near(dx, ref, tol)
    near(dw, rw, tw)
    near(db, rb, tb)


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 8), (40, 16), (1, 64), (133, 100), (7, 513), (300, 768), (9, 1000), (2500, 24),
          (61, 1999), (17, 3584), (701, 4096), (5, 5120), (4, 6200), (3, 8192), (2, 12296), (3, 16384), (2, 16383)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n, d", SHAPES)
def test_norm_and_its_gradient(n, d, dtype):
    rng = np.random.default_rng(n * 131 + d)
    x, dy = make(rng, (n, d), dtype, 1.5, 0.3), make(rng, (n, d), dtype)
    w, b = make(rng, d, dtype, 0.2, 1.0), make(rng, d, dtype, 0.2)
    check(x, dy, w if n % 2 else None, b if d % 2 else None)
    check(x, dy, w, b)


@pytest.mark.parametrize("rows", [152 * 3, 152 * 3 + 1, 20000])
@pytest.mark.parametrize("d", [32, 256, 2048])
def test_more_rows_than_a_pass_of_the_device(rows, d):
    rng = np.random.default_rng(rows + d)
    check(make(rng, (rows, d), "bf16"), make(rng, (rows, d), "bf16"), make(rng, d, "bf16", 0.2, 1), make(rng, d, "bf16"))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows, d", [(3001, 1999), (2000, 513), (5000, 37), (9000, 9), (1000, 4099), (1000, 4098), (700, 8191),
                                     (400, 12289), (400, 16381), (400, 16383), (1, 16383), (153, 6004)])
def test_odd_widths(rows, d, dtype):
    """Rows that begin at every distance from a 16-byte boundary, over many steps."""
    rng = np.random.default_rng(rows + d)
    x, dy = make(rng, (rows, d), dtype, 1.5, 0.3), make(rng, (rows, d), dtype)
    w, b = make(rng, d + 1, dtype, 0.2, 1.0), make(rng, d + 1, dtype, 0.2)
    check(x, dy, w[:d], b[1:])
    flat = make(rng, rows * (d + 2) + 8, dtype)
    part = lambda: flat.as_strided((rows, d), (d + 2, 1), 3)  # (all begin alike, at no boundary)
    check(part(), part().clone(), w[1:], None)
    guard = torch.full((rows * (d + 2) + 8,), 7.0, device="cuda").to(TYPES[dtype])
    y = guard.as_strided((rows, d), (d + 2, 1), 3)
    with norm.NormPlan(d=d, dtype=dtype) as plan:
        plan.forward(part(), y, w[1:])
        near(y, *forward(f64(part()), f64(w[1:]), 0.0, 1e-5))
        plan.backward(part(), part(), y, w[1:])
        near(y, *backward(f64(part()), f64(part()), f64(w[1:]), 1e-5)[:2])
    keep = torch.ones_like(guard, dtype=torch.bool)
    keep.as_strided((rows, d), (d + 2, 1), 3).fill_(False)
    assert (guard[keep] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [96, 4096])
def test_strides_and_alignment(d, dtype):
    """Rows inside wider ones, rows and vectors that are not 16-byte aligned, in place, overlapping input rows."""
    rng = np.random.default_rng(d)
    wide = lambda extra, at: make(rng, (33, d + extra), dtype)[:, at:at + d]
    w, b = make(rng, d + 1, dtype, 0.2, 1.0), make(rng, d + 1, dtype)
    for extra, at in ((8, 0), (8, 8), (3, 0), (3, 1), (8, 4)):
        check(wide(extra, at), wide(0, 0), w[:d], b[:d])
        check(wide(0, 0), wide(extra, at), w[:d], b[:d])
        check(wide(extra, at), wide(extra, at), w[:d], b[:d], inplace=True)
    check(wide(0, 0), wide(0, 0), w[1:], b[1:])
    flat = make(rng, 5 * 32 + d, dtype)
    check(flat.as_strided((6, d), (32, 1)), make(rng, (6, d), dtype), w[:d], None)
    check(flat.as_strided((6, d), (0, 1)), make(rng, (6, d), dtype), w[:d], None)


def test_outputs_in_wider_rows_leave_the_rest():
    rng = np.random.default_rng(5)
    x, dy = make(rng, (50, 264), "bf16"), make(rng, (50, 264), "bf16")
    y, dx = torch.full((50, 300), 7.0, device="cuda").bfloat16(), torch.full((50, 300), 7.0, device="cuda").bfloat16()
    with norm.NormPlan(d=264) as plan:
        plan.forward(x, y[:, 8:272])
        plan.backward(x, dy, dx[:, 8:272])
    near(y[:, 8:272].contiguous(), *forward(f64(x), np.ones(264), np.zeros(264), 1e-5))
    near(dx[:, 8:272].contiguous(), *backward(f64(x), f64(dy), np.ones(264), 1e-5)[:2])
    for t in (y, dx):
        assert (t[:, :8] == 7).all() and (t[:, 272:] == 7).all()


@pytest.mark.parametrize("shift, scale", [(1000.0, 1.0), (0.0, 1e-4), (-3e4, 10.0), (0.0, 1e4)])
def test_means_and_scales(shift, scale):
    """A large mean, rows of the size of eps's root, large rows."""
    rng = np.random.default_rng(3)
    check(make(rng, (37, 1024), "fp32", scale, shift), make(rng, (37, 1024), "fp32"), make(rng, 1024, "fp32", 0.2, 1), None)


def test_constant_rows():
    """No deviation at all: y = b, dx = (g - mean g) / sqrt(eps)."""
    x = torch.full((9, 256), 3.0, device="cuda")
    rng = np.random.default_rng(3)
    w, b, dy = make(rng, 256, "fp32"), make(rng, 256, "fp32"), make(rng, (9, 256), "fp32")
    check(x, dy, w, b)
    with norm.NormPlan(d=256, dtype="fp32") as plan:
        y = torch.empty_like(x)
        plan.forward(x, y, w, b)
        assert torch.equal(y, b.expand_as(y))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 4096, 999])
def test_a_row_that_is_not_finite(d, bad):
    rng = np.random.default_rng(d)
    x, dy = make(rng, (21, d), "bf16"), make(rng, (21, d), "bf16")
    with norm.NormPlan(d=d) as plan:
        want, dwant = torch.empty_like(x), torch.empty_like(x)
        plan.forward(x, want)
        plan.backward(x, dy, dwant)
        x[4, d // 2] = bad
        y, dx = torch.empty_like(x), torch.empty_like(x)
        dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        plan.forward(x, y)
        plan.backward(x, dy, dx, None, dw, db)
    rest = [i for i in range(21) if i != 4]
    assert torch.equal(y[rest], want[rest]) and torch.equal(dx[rest], dwant[rest])
    assert y[4].isnan().all() and dx[4].isnan().all() and dw.isnan().all() and db.isfinite().all()


def test_no_rows_and_partial_gradients():
    with norm.NormPlan(d=40) as plan:
        x = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
        dw, db = torch.full((40,), 7.0, device="cuda"), torch.full((40,), 7.0, device="cuda")
        plan.forward(x, x.clone())
        plan.backward(x, x, x.clone(), None, dw, db)
        assert (dw == 0).all() and (db == 0).all()
        rng = np.random.default_rng(3)
        x, dy = make(rng, (30, 40), "bf16"), make(rng, (30, 40), "bf16")
        dx = [torch.empty_like(x) for _ in range(4)]
        w0, b0 = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
        plan.backward(x, dy, dx[0], None, dw, db)
        plan.backward(x, dy, dx[1], None, w0, None)
        plan.backward(x, dy, dx[2], None, None, b0)
        plan.backward(x, dy, dx[3])
        assert all(torch.equal(dx[0], t) for t in dx[1:]) and torch.equal(w0, dw) and torch.equal(b0, db)


def test_graphs_streams_and_repeats_give_the_same_bits():
    rng = np.random.default_rng(11)
    x, dy = make(rng, (5000, 1032), "bf16"), make(rng, (5000, 1032), "bf16")
    w, b = make(rng, 1032, "bf16"), make(rng, 1032, "bf16")
    new = lambda: (torch.empty_like(x), torch.empty_like(x), torch.empty(1032, device="cuda"), torch.empty(1032, device="cuda"))
    with norm.NormPlan(d=1032) as plan:
        def step(o):
            plan.forward(x, o[0], w, b)
            plan.backward(x, dy, o[1], w, o[2], o[3])

        want, got = new(), new()
        step(want)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(got)
        side.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(got)
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(want, got))


def test_rows_further_apart_than_32_bits_count():
    rng = np.random.default_rng(21)
    far = torch.empty(2 ** 32 + 600, dtype=torch.bfloat16, device="cuda")
    for at in (0, 3):
        x, dy = far.as_strided((3, 520), (2 ** 31, 1), at), make(rng, (3, 520), "bf16")
        x.copy_(make(rng, (3, 520), "bf16"))
        check(x, dy if at == 0 else far.as_strided((3, 520), (2 ** 31, 1), at), make(rng, 520, "bf16"), None)
        y = far.as_strided((3, 520), (2 ** 31, 1), at)
        x = make(rng, (3, 520), "bf16")
        with norm.NormPlan(d=520) as plan:
            plan.forward(x, y)
        near(y, *forward(f64(x), np.ones(520), np.zeros(520), 1e-5))


@pytest.mark.parametrize("d", [520, 1003])
def test_rows_behind_the_last_one_are_left(d):
    rng = np.random.default_rng(22)
    x, dy = make(rng, (900, d), "bf16"), make(rng, (900, d), "bf16")
    x[700:], dy[700:] = float("nan"), float("inf")
    y, dx = torch.full_like(x, 7), torch.full_like(x, 7)
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    with norm.NormPlan(d=d) as plan:
        plan.forward(x[:700], y[:700])
        plan.backward(x[:700], dy[:700], dx[:700], None, dw, db)
    assert (y[700:] == 7).all() and (dx[700:] == 7).all()
    ref, tol, (rw, tw), (rb, tb) = backward(f64(x[:700]), f64(dy[:700]), np.ones(d), 1e-5)
    near(y[:700], *forward(f64(x[:700]), np.ones(d), np.zeros(d), 1e-5))
    near(dx[:700], ref, tol)
    near(dw, rw, tw)
    near(db, rb, tb)


def test_refused_calls():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    f = torch.zeros(64, device="cuda")
    with norm.NormPlan(d=64) as plan:
        for call in (lambda: plan.forward(x.float(), x), lambda: plan.forward(x[:, :32], x), lambda: plan.forward(x, x[:3]),
                     lambda: plan.forward(x.cpu(), x), lambda: plan.forward(x, x, f), lambda: plan.forward(x, x, x[0, :32]),
                     lambda: plan.forward(x.t().contiguous().t(), x), lambda: plan.backward(x, x, x, None, x[0]),
                     lambda: plan.backward(x, x, x, None, f[:32]), lambda: plan.forward(x[None], x[None])):
            with pytest.raises(ValueError):
                call()
        # status from the library: overlapping outputs, a bad eps
        for call in (lambda: plan.forward(x, x[:1].expand(4, 64)), lambda: plan.backward(x, x, x[:1].expand(4, 64)),
                     lambda: plan.forward(x, x, eps=-1.0), lambda: plan.forward(x, x, eps=float("nan")),
                     lambda: plan.backward(x, x, x, eps=float("inf"))):
            with pytest.raises(syn.SynError) as e:
                call()
            assert e.value.status == syn.ERR_INVALID
    for kw, status in ((dict(d=0), syn.ERR_INVALID), (dict(d=16385), syn.ERR_UNSUPPORTED)):
        with pytest.raises(syn.SynError) as e:
            norm.NormPlan(**kw)
        assert e.value.status == status


def test_outputs_in_the_place_of_other_operands_are_refused():
    """In place is with the same stride; dw and db are two vectors."""
    n, d = 4, 64
    wide = torch.zeros(n, 2 * d, dtype=torch.bfloat16, device="cuda")
    x, narrow = wide[:, :d], wide.view(-1)[:n * d].view(n, d)  # (both begin in one place)
    other, f = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(d, device="cuda")
    with norm.NormPlan(d=d) as plan:
        for call in (lambda: plan.forward(x, narrow), lambda: plan.backward(x, other, narrow), lambda: plan.backward(other, x, narrow),
                     lambda: plan.backward(x, other, x, dw=f, db=f)):
            with pytest.raises(syn.SynError) as e:
                call()
            assert e.value.status == syn.ERR_INVALID
        plan.forward(x, x)
        plan.forward(x[:1], narrow[:1])
        plan.backward(x, other, x, dw=f, db=torch.zeros_like(f))
        plan.backward(other, x, x, dw=f)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows, d, apart", [(8003, 777, 777), (9001, 777, 780), (20011, 333, 335), (5003, 1999, 1999), (3001, 4099, 4101)])
def test_in_place_over_many_steps(rows, d, apart, dtype):
    """Rows that begin at no 16-byte boundary, so many that blocks take them in steps: a row's
    first and last vectors are read with a neighbour's elements beside them while that row is
    written.  The same bits as in other tensors that lie alike, whose values are checked; what
    lies between and around the rows stays."""
    rng = np.random.default_rng(rows + d)
    size = rows * apart + 16
    part = lambda t: t.as_strided((rows, d), (apart, 1), 3)
    flat = lambda: make(rng, size, dtype, 1.5, 0.3)
    x, dy = flat(), flat()
    w, b = make(rng, d, dtype, 0.2, 1.0), make(rng, d, dtype, 0.2)
    keep = torch.ones(size, dtype=torch.bool, device="cuda")
    part(keep).fill_(False)
    sums = lambda: [torch.full((d,), 7.0, device="cuda") for _ in range(2)]
    with norm.NormPlan(d=d, dtype=dtype) as plan:
        y, dx, dsum = torch.zeros_like(x), torch.zeros_like(x), sums()
        plan.forward(part(x), part(y), w, b)
        plan.backward(part(x), part(dy), part(dx), w, *dsum)
        x0, g0, w0 = f64(part(x)), f64(part(dy)), f64(w)
        near(part(y), *forward(x0, w0, f64(b), 1e-5))
        ref, tol, (rw, tw), (rb, tb) = backward(x0, g0, w0, 1e-5)
        near(part(dx), ref, tol)
        near(dsum[0], rw, tw)
        near(dsum[1], rb, tb)
        for _ in range(5):
            over, over_dy, over_x, s1, s2 = x.clone(), dy.clone(), x.clone(), sums(), sums()
            plan.forward(part(over), part(over), w, b)
            plan.backward(part(x), part(over_dy), part(over_dy), w, *s1)
            plan.backward(part(over_x), part(dy), part(over_x), w, *s2)
            for got, want, before in ((over, y, x), (over_dy, dx, dy), (over_x, dx, x)):
                assert torch.equal(part(got), part(want)) and torch.equal(got[keep], before[keep])
            assert all(torch.equal(p, q) for s in (s1, s2) for p, q in zip(s, dsum))
