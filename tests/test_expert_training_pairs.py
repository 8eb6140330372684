"""The CTA pairs of moe_expert_project and its backward pass: sums that several of them share, the limit of their
waits.  Beside test_expert_training.py, whose cases, definitions and tolerances these tests take."""
import numpy as np
import pytest
import torch

import moe_expert_layer_06_gb300 as m
from test_expert_training import BF, F32, Case, close


def slots_of(c):
    """The rows of each slot as the header has them cut: from its offset to the next one, none where that is lower."""
    lo = np.clip(c.off[:-1], 0, c.R)
    return [slice(int(a), int(max(a, b))) for a, b in zip(lo, np.clip(c.off[1:], 0, c.R))]


def by_slot(c):
    """For each slot with rows: (rows, (y, tolerance), (dx, tolerance)); and every slot's [(dw, tolerance)], all in fp64."""
    rows, dw = [], []
    for s, r in enumerate(slots_of(c)):
        one = Case(c.R, c.K, c.N, 1, c.P, [0, 0])
        one.x, one.dy, one.w = c.x[r], c.dy[r], [w[s:s + 1] for w in c.w]
        one.R, one.off = r.stop - r.start, np.asarray([0, r.stop - r.start], dtype=np.int32)
        y, dx, (g, eg) = one.reference()
        dw.append([(a[0], b[0]) for a, b in zip(g, eg)])
        if one.R:
            rows.append((r, y, dx))
    return rows, dw


def within(got, want, tol):
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -23
    return (got.double().cpu() - want).abs() <= tol + half * (want.abs() + tol) + 1e-30


# Offsets that run backwards name rows several times: more tiles than offsets in order give.  Each value is that of
# one of its row's slots, and each slot's dw that of its rows; the same where pairs would share the sums.
@pytest.mark.gpu
@pytest.mark.parametrize("K,N,P", [(1024, 256, 1), (256, 1024, 1), (256, 520, 2), (2056, 72, 2), (72, 2056, 1)])
def test_offsets_that_run_backwards(K, N, P):
    c = Case(2560, K, N, 5, P, [0, 2000, 0, 2000, 0, 2560], seed=30)
    rows, dw = by_slot(c)

    def check(got, which, name):
        fits = torch.zeros(got.shape, dtype=torch.bool)
        for r, *values in rows:
            fits[r] |= within(got[r], *values[which])
        assert bool(fits.all()), (name, int((~fits).sum()))

    for dtype in (BF, F32):
        check(c.forward(dtype), 0, "y")
        check(c.backward(dw=False, dx_type=dtype)[0], 1, "dx")
        both, alone = c.backward(dx_type=dtype, dw_type=dtype), c.backward(dx=False, dw_type=dtype)
        check(both[0], 1, "dx beside dw")
        for s in range(5):
            for p in range(P):
                close(both[1][p][s], *dw[s][p], name=f"dw{p} of slot {s}")
                close(alone[1][p][s], *dw[s][p], name=f"dw{p} of slot {s} alone")
    assert m.moe_check_status() == m.MOE_ERR_DEVICE_STATUS


@pytest.mark.gpu
def test_a_limit_of_the_waits_below_the_time_of_a_call():
    """The limit is of each wait, not of the kernel: calls of some milliseconds give the same bits under 0.5 ms."""
    R, K, N, S = 32768, 7168, 2048, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF)  # noqa: E731
    p, off = m.Project(K, N, S, 2), torch.linspace(0, R, S + 1, device="cuda").round().to(torch.int32)
    x, dy, w, w2 = new(R, K), new(R, 2 * N), new(S, N, K), new(S, N, K)
    codes, scale = torch.empty(R, K, dtype=torch.uint8, device="cuda"), torch.empty(R, K // 128, device="cuda")
    m.moe_checkpoint_rows(R, K, x, codes, scale)

    def step():
        y, dx = torch.empty(R, 2 * N, dtype=BF, device="cuda"), torch.empty(R, K, dtype=BF, device="cuda")
        dw = [torch.empty(S, N, K, dtype=BF, device="cuda") for _ in range(4)]
        m.moe_expert_project(p, R, x, off, w, w2, y)
        m.moe_expert_project_backward(p, R, dy, x, None, None, off, w, w2, dx, *dw[:2])
        m.moe_expert_project_backward(p, R, dy, None, codes, scale, off, None, None, None, *dw[2:])
        return [y, dx, *dw]

    want = step()
    assert m.moe_check_status() == m.MOE_OK
    m.moe_set_wait_limit_ns(500_000)
    try:
        got = step()
        assert m.moe_check_status() == m.MOE_OK
    finally:
        m.moe_set_wait_limit_ns(2_000_000_000)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
