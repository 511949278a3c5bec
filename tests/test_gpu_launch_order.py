"""The rotary and windowed-attention operators behind the fused GEMM that makes
their rows, whose CTAs let the next kernel of the stream start at their own
beginning: the same bits without any synchronisation between the calls as with
one after each of them."""
import numpy as np
import pytest
import torch

from chunk_scheduled_communication_gb300 import rope, runner, syn, window
from chunk_scheduled_communication_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
H_Q, H_KV, D, TOKENS, SETS = 4, 2, 128, 2048, 3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    syn.lib()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("backend, tile_m", [("tma_colocated", 256), ("tma_colocated", 128), ("tma_dedicated", 256)])
def test_projection_rotation_attention(backend, tile_m, norm):
    w = wl.scaled(wl.TINY_AG, M=TOKENS, K=1024, N=(H_Q + 2 * H_KV) * D, R=2)
    sets = [runner.upload(wl.make_inputs(w, r=1, seed=s)) for s in range(SETS)]
    qkv = torch.empty((TOKENS, H_Q + 2 * H_KV, D), dtype=torch.bfloat16, device="cuda")  # of every call in turn
    for d in sets:
        d.out = qkv.view(TOKENS, -1)
    q, k, v = qkv[:, :H_Q], qkv[:, H_Q:H_Q + H_KV], qkv[:, H_Q + H_KV:]
    qr, kr, vr = (torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k, v))
    back = [torch.empty_like(t) for t in (qr, kr)]
    out, out2 = torch.empty_like(qr), torch.empty_like(qr)
    g = torch.Generator(device="cuda").manual_seed(1)
    pos = torch.randint(0, 100000, (TOKENS,), generator=g, device="cuda")
    weight = torch.randn(D, generator=g, device="cuda").bfloat16()
    kept = [torch.empty_like(t) for t in (qr, kr, vr, *back, out, out2, qkv)]
    lens = [TOKENS - 700, 700]
    gemm = runner.make_plan(sets[0], split=2, order="row", backend=backend, tile_m=tile_m, comm_sms=4)
    with gemm, rope.RopePlan() as turn, \
            window.WindowPlan(lens, H_q=H_Q, H_kv=H_KV, window=100, sinks=4) as plan:

        def calls(d, pause):
            """Every call reads what the one before wrote, and overwrites what the round before read."""
            def rotate(q, q_out, k, k_out, *more):
                if norm:
                    turn.norm_rotate(q, q_out, weight, k, k_out, weight, *more, positions=pos)
                else:
                    turn.rotate(q, q_out, k, k_out, *more, positions=pos)

            runner.call(gemm, d)                # qkv
            pause()
            rotate(q, qr, k, kr, v, vr)         # into other rows, V copied
            pause()
            runner.call(gemm, d)                # the same again, over rows that were just read
            pause()
            turn.rotate_backward(q, back[0], k, back[1], positions=pos)
            pause()
            plan.forward(qr, kr, v, out)        # V as the GEMM left it
            pause()
            rotate(q, q, k, k)                  # in place
            pause()
            plan.forward(q, k, v, out2)
            pause()

        def result(d, pause, into):
            calls(d, pause)
            for a, b in zip(into, (qr, kr, vr, *back, out, out2, qkv)):
                a.copy_(b)
            pause()
            return into

        want = [result(d, torch.cuda.synchronize, [torch.empty_like(t) for t in kept]) for d in sets]
        assert all(t.isfinite().all() for t in want[0])
        assert not torch.equal(want[0][0], want[1][0])
        rng = np.random.default_rng(2)
        for _ in range(40):
            i = int(rng.integers(SETS))
            got = result(sets[i], lambda: None, kept)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        gemm.check()
        plan.check()
