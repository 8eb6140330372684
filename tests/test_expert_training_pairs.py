"""The CTA pairs of moe_expert_project and its backward pass: sums that several of them share, the limit of their
waits.  Beside test_expert_training.py, whose cases, definitions and tolerances these tests take."""
import numpy as np
import pytest
import torch

import moe_expert_layer_06_gb300 as m
from test_expert_training import BF, F32, HALF, STEP, Case, close, ragged


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


Y, DX, DW, ROWS8 = 0, m.MOE_PLAN_DX, m.MOE_PLAN_DW, m.MOE_PLAN_ROWS8


def codes_of(c, seed):
    """(codes, scales, the values they stand for): every code, the scale of a row any power of two."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (c.R, c.K), generator=g).to(torch.uint8)
    codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes)
    scales = torch.exp2(torch.randint(-12, 4, (c.R, -(-c.K // 128)), generator=g).float())
    return codes, scales, (codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)[:, :c.K]).to(BF)


# Every way in which sums are shared, alone and side by side in one launch; the plan is asked for, so that sizes which
# another rule would run otherwise show here.  (R, K, N, slots, parts), outputs, plan.
PLANS = [
    ((394, 1008, 8, 5, 2), Y, (2, 0, 0, 0)), ((300, 1096, 1000, 2, 2), Y, (2, 0, 0, 0)), ((4, 1088, 72, 1, 1), Y, (4, 0, 0, 0)),
    ((449, 304, 1024, 5, 1), DX, (2, 0, 0, 0)), ((40, 2280, 824, 3, 2), DX, (2, 0, 0, 0)), ((46, 16, 1120, 2, 1), DX, (4, 0, 0, 0)),
    ((1483, 800, 312, 1, 2), DW, (0, 2, 0, 0)), ((3815, 1328, 8, 2, 2), DW, (0, 2, 0, 0)), ((2283, 16, 16, 2, 2), DW, (0, 4, 0, 0)),
    ((1401, 576, 376, 1, 2), DX | DW, (1, 2, 1, 0)), ((2283, 16, 16, 2, 2), DX | DW, (1, 4, 1, 0)),
    ((263, 16, 1072, 8, 1), DX | DW, (2, 1, 1, 0)), ((1367, 544, 464, 1, 2), DX | DW, (2, 2, 1, 0)),
    ((1066, 320, 968, 1, 1), DX | DW, (2, 4, 1, 0)), ((46, 16, 1120, 2, 1), DX | DW, (4, 1, 1, 0)),
    ((1371, 96, 1048, 1, 2), DX | DW, (4, 2, 1, 0)), ((967, 16, 520, 1, 2), DX | DW, (4, 4, 1, 0)),
    ((1483, 800, 312, 1, 2), DW | ROWS8, (0, 2, 0, 0)), ((2283, 16, 16, 2, 2), DW | ROWS8, (0, 4, 0, 0)),
    ((1976, 800, 24, 2, 2), DX | DW | ROWS8, (1, 2, 1, 0)), ((2283, 16, 16, 2, 2), DX | DW | ROWS8, (1, 4, 1, 0)),
    ((263, 16, 1072, 8, 1), DX | DW | ROWS8, (2, 1, 1, 0)), ((1056, 544, 1040, 1, 1), DX | DW | ROWS8, (2, 2, 1, 0)),
    ((1066, 320, 968, 1, 1), DX | DW | ROWS8, (2, 4, 1, 0)), ((46, 16, 1120, 2, 1), DX | DW | ROWS8, (4, 1, 1, 0)),
    ((961, 16, 1544, 1, 2), DX | DW | ROWS8, (4, 2, 1, 0)), ((967, 16, 520, 1, 2), DX | DW | ROWS8, (4, 4, 1, 0))]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,outputs,plan", PLANS)
def test_every_plan_of_shared_sums(sizes, outputs, plan):
    c = Case(*sizes, seed=32)
    assert m.moe_debug_project_plan(c.p, c.R, outputs) == plan
    eight, x = None, c.x
    if outputs & ROWS8:
        *eight, x = codes_of(c, 33)
    y, dx, dw = c.reference(x)
    if outputs == Y:
        close(c.forward(), *y, name="y")
        close(c.forward(F32), *y, name="y fp32")
        out = torch.full((c.R, c.P * c.N), 2.0, device="cuda")
        c.forward(F32, add=True, out=out)
        there = ~torch.isnan(y[0])
        close(out, torch.where(there, y[0] + 2.0, 2.0), torch.where(there, y[1] + STEP * (y[0].abs() + 2.0), 0.0), name="y added")
        assert torch.equal(c.forward().nan_to_num(9.0), c.forward().nan_to_num(9.0))
        assert m.moe_check_status() == 0
        return
    want_x, want_w = bool(outputs & DX), bool(outputs & DW)
    for dtype in (BF, F32):
        got = c.backward(want_x, want_w, dtype, dtype, eight)
        again = c.backward(want_x, want_w, dtype, dtype, eight)
        if want_x:
            close(got[0], *dx, name="dx")
            assert torch.equal(got[0].nan_to_num(9.0), again[0].nan_to_num(9.0))
        for p in range(c.P if want_w else 0):
            close(got[1][p], dw[0][p], dw[1][p], name=f"dw{p}")
            assert torch.equal(got[1][p], again[1][p])
    got = c.backward(want_x, want_w, F32, F32, eight, want_x, want_w, fill=1.0)
    if want_x:
        there = ~torch.isnan(dx[0])
        close(got[0], torch.where(there, dx[0] + 1.0, 1.0), torch.where(there, dx[1] + STEP * (dx[0].abs() + 1.0), 0.0), name="dx added")
    for p in range(c.P if want_w else 0):
        close(got[1][p], dw[0][p] + 1.0, dw[1][p] + STEP * (dw[0][p].abs() + 1.0), name=f"dw{p} added")
    assert m.moe_check_status() == 0


# A captured call takes the counts of its replay (shares without a row, a slot that loses all of its rows), and gives the
# same bits beside another on a second stream.
@pytest.mark.gpu
@pytest.mark.parametrize("sizes,alone,both", [((3000, 144, 200, 3, 2), 4, (1, 4, 1, 0)), ((3100, 800, 24, 2, 2), 2, (1, 2, 1, 0)),
                                              ((1066, 320, 968, 1, 1), 4, (2, 4, 1, 0)), ((1371, 96, 1048, 1, 2), 4, (4, 2, 1, 0))])
def test_shared_sums_replayed_with_other_counts(sizes, alone, both):
    c = Case(*sizes, seed=34)
    R, K, N, S, P = sizes
    assert m.moe_debug_project_plan(c.p, R, DW)[1] == alone and m.moe_debug_project_plan(c.p, R, DX | DW) == both
    *eight, values = codes_of(c, 35)
    x, dy, off, (w, w2), (x8, scale) = c.x.cuda(), c.dy.cuda(), c.offsets(), c.weights(), [t.cuda() for t in eight]

    def outputs():
        return [torch.zeros(R, K, dtype=BF, device="cuda")] + [torch.zeros_like(w) if p < P else None for _ in range(3) for p in range(2)]

    def step(dx, dw, dw2, lone, lone2, lone8, lone8_2):
        m.moe_expert_project_backward(c.p, R, dy, x, None, None, off, w, w2, dx, dw, dw2)
        m.moe_expert_project_backward(c.p, R, dy, x, None, None, off, None, None, None, lone, lone2)
        m.moe_expert_project_backward(c.p, R, dy, None, x8, scale, off, None, None, None, lone8, lone8_2)

    graph, side, replayed = torch.cuda.CUDAGraph(), torch.cuda.Stream(), outputs()
    step(*outputs())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(*replayed)
    for counts in (c.off, [0] * S + [R], [0] * S + [65], [0] + [R - 130] * S, [0] * (S + 1), c.off):
        c.off = np.asarray(counts, dtype=np.int32)
        off.copy_(torch.from_numpy(c.off))
        _, dx, dw = c.reference()
        dw8 = c.reference(values)[2]
        graph.replay()
        torch.cuda.synchronize()
        rows = ~torch.isnan(dx[0][:, 0])
        close(replayed[0][rows.cuda()], dx[0][rows], dx[1][rows], name="dx")
        for p in range(P):
            close(replayed[1 + p], dw[0][p], dw[1][p], name=f"dw{p}")
            close(replayed[3 + p], dw[0][p], dw[1][p], name=f"dw{p} alone")
            close(replayed[5 + p], dw8[0][p], dw8[1][p], name=f"dw{p} of codes")
        here, there = outputs(), outputs()
        torch.cuda.synchronize()
        for _ in range(5):
            step(*here)
            with torch.cuda.stream(side):
                step(*there)
        torch.cuda.synchronize()
        for got in (here, there):
            for a, b in zip(got, replayed):
                assert a is None or torch.equal(a[rows.cuda()] if a.shape[0] == R else a, b[rows.cuda()] if b.shape[0] == R else b)
    assert m.moe_check_status() == 0


@pytest.mark.gpu
def test_the_plan_of_a_call():
    p = m.Project(7168, 2048, 32, 2)
    assert m.moe_debug_project_plan(p, 32768) == (1, 0, 0, 0)
    assert m.moe_debug_project_plan(p, 32768, DX | DW | ROWS8) == (1, 1, 0, 1)
    assert m.moe_debug_project_plan(m.Project(328, 600, 16), 100, DX | DW) == (1, 1, 1, 0)
    assert m.moe_debug_project_plan(p, 4096, DX)[1] == 0 and m.moe_debug_project_plan(p, 4096, DW)[0] == 0


def test_plans_that_are_refused():
    p = m.Project(64, 64, 4)
    for args in ((p, 0), (p, -1), (p, 4, -1), (p, 4, 8), (p, 4, ROWS8), (m.Project(60, 64, 4), 4), (m.Project(64, 64, 0), 4)):
        with pytest.raises(m.MoeError):
            m.moe_debug_project_plan(*args)
    assert m.lib().moe_debug_project_plan(None, 4, 0, None) == m.MOE_ERR_INVALID_ARG


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


@pytest.mark.gpu
@pytest.mark.parametrize("R", [37, 4096, 12321])
def test_products_at_the_width_of_a_large_layer(R):
    """7168 to gate and up of 2048 for 32 slots, 2048 to 7168 for the way back: slots with the most and the fewest rows and one
    without any, all of their outputs against fp64."""
    S, H, I = 32, 7168, 2048
    off = ragged(R, S, seed=40)
    counts = np.diff(off)
    some = counts > 0
    look = {int(np.argmax(counts)), int(np.argmin(np.where(some, counts, R + 1))), int(np.argmin(counts))}
    g = torch.Generator(device="cuda").manual_seed(R)
    for K, N, P in ((H, I, 2), (I, H, 1)):
        new = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF)  # noqa: E731
        p, offsets = m.Project(K, N, S, P), torch.from_numpy(off).cuda()
        x, dy, w = new(R, K), new(R, P * N), [new(S, N, K, std=K ** -0.5) for _ in range(P)]
        codes, scale = torch.empty(R, K, dtype=torch.uint8, device="cuda"), torch.empty(R, K // 128, device="cuda")
        m.moe_checkpoint_rows(R, K, x, codes, scale)
        kept = (codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(128, 1)).to(BF)
        y, dx = torch.empty(R, P * N, dtype=BF, device="cuda"), torch.empty(R, K, dtype=BF, device="cuda")
        dw, dw8 = ([torch.full((S, N, K), float("nan"), dtype=BF, device="cuda") for _ in range(P)] for _ in range(2))
        m.moe_expert_project(p, R, x, offsets, *(w + [None])[:2], y)
        m.moe_expert_project_backward(p, R, dy, x, None, None, offsets, *(w + [None])[:2], dx, *dw)
        m.moe_expert_project_backward(p, R, dy, None, codes, scale, offsets, None, None, None, *dw8)
        assert m.moe_check_status() == 0

        def near(got, want, tol):
            assert bool(((got.double() - want).abs() <= tol + HALF * (want.abs() + tol) + 1e-30).all())

        for s in look:
            rows, n = slice(int(off[s]), int(off[s + 1])), int(counts[s])
            a, want, bound = x[rows].double(), 0.0, 0.0
            for q in range(P):
                cols, ws, d = slice(q * N, (q + 1) * N), w[q][s].double(), dy[rows, q * N:(q + 1) * N].double()
                near(y[rows, cols], a @ ws.t(), K * STEP * (a.abs() @ ws.abs().t()))
                want, bound = want + d @ ws, bound + P * N * STEP * (d.abs() @ ws.abs())
                for rows_of, got in ((a, dw[q][s]), (kept[rows].double(), dw8[q][s])):
                    near(got, d.t() @ rows_of, n * STEP * (d.abs().t() @ rows_of.abs()))
            near(dx[rows], want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(1 << 24, 8), (8, 1 << 24)])
def test_the_most_features(K, N):
    """2^24 on either side: sums of -1, 0 and 1, which are whole numbers below 2^8 and so exact in bf16, too."""
    R, S = 5, 2
    g = torch.Generator(device="cuda").manual_seed(K)
    few = lambda *s: torch.where(torch.rand(*s, generator=g, device="cuda") < 1e-4,  # noqa: E731
                                 torch.randint(0, 2, s, generator=g, device="cuda") * 2.0 - 1.0, 0.0)
    many = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda").float()  # noqa: E731
    x, dy, w = (few if K > N else many)(R, K), (many if K > N else few)(R, N), many(S, N, K)
    off = [0, 2, 4]  # (the last row is of no slot)
    p, offsets = m.Project(K, N, S), torch.tensor(off, dtype=torch.int32, device="cuda")
    y, dx, dw = (torch.full(s, 7.0, dtype=BF, device="cuda") for s in ((R, N), (R, K), (S, N, K)))
    m.moe_expert_project(p, R, x.to(BF), offsets, w.to(BF), None, y)
    m.moe_expert_project_backward(p, R, dy.to(BF), x.to(BF), None, None, offsets, w.to(BF), None, dx, dw)
    assert m.moe_check_status() == 0
    for s in range(S):
        rows = slice(off[s], off[s + 1])
        for got, a, b in ((y[rows], x[rows], w[s].t()), (dx[rows], dy[rows], w[s]), (dw[s], dy[rows].t(), x[rows])):
            want = a.double() @ b.double()
            assert float(want.abs().max()) < 256 and torch.equal(got.double(), want)
    assert bool((y[4] == 7.0).all()) and bool((dx[4] == 7.0).all())
