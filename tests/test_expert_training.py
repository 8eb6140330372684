"""The operators that train the experts (moe_expert_project and its backward pass, activations kept
in 8 bits, SwiGLU on them, the combine's gradient) against their definitions in 64 bits.

Tolerances, element by element.  An output rounds once (bf16: half a step, 2^-8 of its value; fp32:
2^-24); an fp32 sum of n products is off by at most n steps of 2^-23 of the sum of their magnitudes
(2^-24 for a rounded sum; twice that where a tensor core truncates).  Codes and scales are equal.
SwiGLU: the sigmoid is 1 / (1 + 2^(-g log2 e)).  log2 e and its product with g are rounded, 2^-24 each of up to
70 * 1.45 (beyond |g| = 70 what it gives is below the 1e-30 that every comparison allows): 71 steps of 2^-23 of
the power; ex2.approx adds 2, the sum half of one, rcp.approx 1 and the few products beside it less than 10:
2^-16 (128 steps) of the factors in all."""
import ctypes

import numpy as np
import pytest
import torch

import moe_expert_layer_06_gb300 as m

FAKE = 0x10000  # aligned address that is never dereferenced on the host
HALF = 2.0 ** -8
STEP = 2.0 ** -23
BF, F32 = torch.bfloat16, torch.float32


def ragged(R, S, seed=0, empty=True):
    """Offsets [S + 1] of R rows in S slots, uneven, some slots without a row."""
    rs = np.random.RandomState(seed + 7 * R + S)
    p = np.exp(rs.randn(S))
    if empty and S > 2:
        p[rs.randint(0, S, max(1, S // 4))] = 0.0
        p[rs.randint(0, S)] += 1e-3
    return np.concatenate([[0], np.cumsum(rs.multinomial(R, p / p.sum()))]).astype(np.int32)


class Case:
    def __init__(self, R, K, N, S, P, offsets=None, seed=0):
        g = torch.Generator().manual_seed(seed + 31 * R + K + N + S)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g) * std).to(BF)

        self.R, self.K, self.N, self.S, self.P = R, K, N, S, P
        self.p = m.Project(K, N, S, P)
        self.off = ragged(R, S, seed) if offsets is None else np.asarray(offsets, dtype=np.int32)
        self.x, self.dy = normal(R, K), normal(R, P * N)
        self.w = [normal(S, N, K, std=K ** -0.5) for _ in range(P)]

    def offsets(self):
        return torch.from_numpy(self.off).cuda()

    def weights(self):
        return [w.cuda() for w in self.w] + [None] * (2 - self.P)

    def forward(self, dtype=BF, add=False, out=None):
        if out is None:
            out = torch.full((self.R, self.P * self.N), float("nan"), dtype=dtype, device="cuda")
        w, w2 = self.weights()
        m.moe_expert_project(self.p, self.R, self.x.cuda(), self.offsets(), w, w2, out, add)
        return out

    def backward(self, dx=True, dw=True, dx_type=BF, dw_type=BF, eight=None, add_dx=False, add_dw=False, fill=float("nan")):
        """(dx, [dw, dw2]); eight: (codes, scale) in the place of x."""
        w, w2 = self.weights()
        dx = torch.full((self.R, self.K), fill, dtype=dx_type, device="cuda") if dx else None
        dws = [torch.full((self.S, self.N, self.K), fill, dtype=dw_type, device="cuda") if dw else None for _ in range(self.P)]
        x8, scale = (None, None) if eight is None else (eight[0].cuda(), eight[1].cuda())
        m.moe_expert_project_backward(self.p, self.R, self.dy.cuda(), self.x.cuda() if eight is None else None, x8, scale,
                                      self.offsets(), w, w2, dx, *(dws + [None])[:2], add_dx, add_dw)
        return dx, dws

    def reference(self, x=None):
        """(y, dx, [dw]) as values and tolerances of their fp32 sums, fp64; y and dx of rows in no slot are NaN."""
        x, dy, P, N = (self.x if x is None else x).double(), self.dy.double(), self.P, self.N
        y, ey = (torch.full((self.R, P * N), float("nan")).double() for _ in range(2))
        dx, edx = (torch.full((self.R, self.K), float("nan")).double() for _ in range(2))
        dw = [torch.zeros_like(w, dtype=torch.float64) for w in self.w]
        edw = [torch.zeros_like(w, dtype=torch.float64) for w in self.w]
        for s in range(self.S):
            rows = slice(int(self.off[s]), int(self.off[s + 1]))
            n = rows.stop - rows.start
            if not n:
                continue
            dx[rows], edx[rows] = 0.0, 0.0
            for p in range(P):
                w, cols = self.w[p][s].double(), slice(p * N, (p + 1) * N)
                y[rows, cols], ey[rows, cols] = x[rows] @ w.t(), self.K * STEP * (x[rows].abs() @ w.abs().t())
                dx[rows] += dy[rows, cols] @ w
                edx[rows] += P * N * STEP * (dy[rows, cols].abs() @ w.abs())
                dw[p][s], edw[p][s] = dy[rows, cols].t() @ x[rows], n * STEP * (dy[rows, cols].abs().t() @ x[rows].abs())
        return (y, ey), (dx, edx), (dw, edw)


def close(got, want, tol, name=""):
    """Rows without a value (NaN) are left as they were (NaN)."""
    half = HALF if got.dtype == BF else 2.0 ** -23
    got = got.double().cpu()
    there = ~torch.isnan(want)
    assert bool(torch.isnan(got[~there]).all()), (name, "rows of no slot were written")
    got, want, tol = got[there], want[there], tol[there]
    tol = tol + half * (want.abs() + tol) + 1e-30
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (name, int(bad.sum()), float(((got - want).abs() / tol).max()))


# (K, N, slots, parts): every size ragged somewhere; a single tile, several, tails of every kind
SIZES = [(8, 8, 1, 1), (64, 128, 3, 2), (72, 136, 5, 1), (600, 328, 16, 2), (256, 512, 2, 1), (520, 264, 7, 2), (1000, 616, 4, 1),
         (328, 1040, 40, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("R", [1, 2, 17, 63, 64, 65, 200, 700])
@pytest.mark.parametrize("K,N,S,P", SIZES)
def test_products_match_the_definition(R, K, N, S, P):
    c = Case(R, K, N, S, P)
    y, dx, dw = c.reference()
    close(c.forward(), *y, name="y")
    got = c.backward()
    assert m.moe_check_status() == 0
    close(got[0], *dx, name="dx")
    for p in range(P):
        close(got[1][p], dw[0][p], dw[1][p], name=f"dw{p}")


@pytest.mark.gpu
@pytest.mark.parametrize("R,K,N,S,P", [(1500, 264, 520, 2, 2), (2100, 136, 72, 1, 1), (1300, 2056, 1032, 3, 1), (900, 72, 2056, 300, 1), (1100, 72, 136, 1024, 2),
                                       (60, 8, 8, 1024, 1)])
def test_many_rows_of_a_slot_and_many_slots(R, K, N, S, P):
    c = Case(R, K, N, S, P, seed=3)
    y, dx, dw = c.reference()
    close(c.forward(), *y, name="y")
    got = c.backward()
    assert m.moe_check_status() == 0
    close(got[0], *dx, name="dx")
    for p in range(P):
        close(got[1][p], dw[0][p], dw[1][p], name=f"dw{p}")


# few tiles of a long contraction, which pairs of CTAs share (from 16 chunks of 64 on: four, or two where there are more
# tiles; test_expert_training_pairs.py asks for the plan of each call)
@pytest.mark.gpu
@pytest.mark.parametrize("R", [1, 5, 70, 300])
@pytest.mark.parametrize("K,N,S,P", [(2056, 136, 1, 1), (4104, 264, 2, 2), (1032, 8, 3, 1), (136, 2056, 2, 1), (264, 1544, 1, 2), (8, 4104, 3, 2)])
def test_long_contractions_of_few_tiles(R, K, N, S, P):
    c = Case(R, K, N, S, P, seed=14)
    y, dx, dw = c.reference()
    for dtype in (BF, F32):
        close(c.forward(dtype), *y, name="y")
        close(c.backward(dw=False, dx_type=dtype)[0], *dx, name="dx")
        got = c.backward(dx_type=dtype)
        close(got[0], *dx, name="dx beside dw")
        for p in range(P):
            close(got[1][p], dw[0][p], dw[1][p], name=f"dw{p}")
    out = torch.full((R, P * N), 2.0, device="cuda")
    c.forward(F32, add=True, out=out)
    there = ~torch.isnan(y[0])
    close(out, torch.where(there, y[0] + 2.0, 2.0), torch.where(there, y[1] + STEP * (y[0].abs() + 2.0), 0.0), name="y added")
    first = c.forward()
    assert torch.equal(first.nan_to_num(9.0), c.forward().nan_to_num(9.0))
    assert m.moe_check_status() == 0
    # rows of the next slot and of none beside it
    if R >= 70:
        c.x[-1, 3], c.dy[-1, 5] = float("inf"), float("nan")
        close(c.forward()[:-1], y[0][:-1], y[1][:-1], name="y beside an infinity")
        close(c.backward(dw=False)[0][:-1], dx[0][:-1], dx[1][:-1], name="dx beside a NaN")


# few tiles of dw with long sums, which pairs of CTAs share too; slots with fewer chunks than pairs, or none
@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[2500], [3000, 0, 70], [1, 2200, 64, 1900], [130, 4000]])
@pytest.mark.parametrize("K,N,P", [(136, 200, 1), (272, 40, 2), (16, 8, 1)])
def test_long_sums_of_few_tiles(counts, K, N, P):
    off = np.concatenate([[0], np.cumsum(counts)])
    c = Case(int(off[-1]) + 9, K, N, len(counts), P, off, seed=15)
    _, dx, dw = c.reference()
    for beside in (False, True):
        for dtype in (BF, F32):
            got = c.backward(dx=beside, dw_type=dtype)
            if beside:
                close(got[0], *dx, name="dx")
            for p in range(P):
                close(got[1][p], dw[0][p], dw[1][p], name=f"dw{p}")
    added = c.backward(dx=False, dw_type=F32, add_dw=True, fill=1.0)[1]
    for p in range(P):
        close(added[p], dw[0][p] + 1.0, dw[1][p] + STEP * (dw[0][p].abs() + 1.0), name=f"dw{p} added")
    if K % 16 == 0:
        g = torch.Generator().manual_seed(K)
        codes = torch.randint(0, 256, (c.R, K), generator=g).to(torch.uint8)
        codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes)
        scales = torch.exp2(torch.randint(-12, 4, (c.R, -(-K // 128)), generator=g).float())
        values = (codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)[:, :K]).to(BF)
        kept_dw = c.reference(values)[2]
        for beside in (False, True):
            got = c.backward(dx=beside, eight=(codes, scales))
            for p in range(P):
                close(got[1][p], kept_dw[0][p], kept_dw[1][p], name=f"dw{p} of codes")
    assert m.moe_check_status() == 0
    # the row behind the last slot, and one of the largest slot: the others' gradients do not see them
    big = int(np.argmax(counts))
    c.x[-1, 3], c.dy[-1, 5] = float("inf"), float("nan")
    c.x[off[big] + 1, 3], c.dy[off[big] + 1, 5] = float("inf"), float("nan")
    got = c.backward(dx=False)[1]
    for s in range(len(counts)):
        if s != big:
            close(got[0][s], dw[0][0][s], dw[1][0][s], name="dw beside infinities")


# shared memory that a call of NaNs left is not seen where a narrow output's copies are left out
@pytest.mark.gpu
@pytest.mark.parametrize("N", [8, 64, 128, 136, 192, 320, 392])
@pytest.mark.parametrize("R,K,S,P", [(700, 328, 2, 1), (30, 2056, 1, 2), (2000, 72, 3, 2)])
def test_narrow_outputs_after_a_call_of_nans(R, K, S, P, N):
    nan = Case(3000, 520, 520, 2, 2, seed=16)
    nan.x.fill_(float("nan"))
    nan.dy.fill_(float("nan"))
    c = Case(R, K, N, S, P, seed=17)
    y, dx, dw = c.reference()
    for dtype in (BF, F32):
        nan.forward()
        close(c.forward(dtype), *y, name="y")
        nan.backward()
        got = c.backward(dx_type=dtype, dw_type=dtype)
        close(got[0], *dx, name="dx")
        for p in range(P):
            close(got[1][p], dw[0][p], dw[1][p], name=f"dw{p}")
        nan.backward()
        got = c.backward(dx=False, dw_type=dtype)[1]
        for p in range(P):
            close(got[p], dw[0][p], dw[1][p], name=f"dw{p} alone")
    assert m.moe_check_status() == 0


# sums that pairs share: a captured call takes the counts of its replay, repeats bit for bit, on two streams too
@pytest.mark.gpu
def test_shared_sums_captured_repeated_and_beside_each_other():
    R, K, N, S = 2600, 144, 200, 3
    c = Case(R, K, N, S, 2, [0, 2000, 2000, 2600], seed=18)
    x, dy, off, (w, w2) = c.x.cuda(), c.dy.cuda(), c.offsets(), c.weights()

    def outputs():
        return [torch.zeros(R, K, dtype=BF, device="cuda")] + [torch.zeros_like(w) for _ in range(4)]

    def step(dx, dw, dw2, alone, alone2):
        m.moe_expert_project_backward(c.p, R, dy, x, None, None, off, w, w2, dx, dw, dw2)
        m.moe_expert_project_backward(c.p, R, dy, x, None, None, off, None, None, None, alone, alone2)

    first = outputs()
    step(*first)
    graph, side, replayed = torch.cuda.CUDAGraph(), torch.cuda.Stream(), outputs()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(*replayed)
    for offsets in ([0, 2000, 2000, 2600], [0, 0, 2600, 2600], [0, 1, 100, 2500]):
        off.copy_(torch.tensor(offsets, dtype=torch.int32))
        c.off = np.asarray(offsets, dtype=np.int32)
        _, dx, dw = c.reference()
        graph.replay()
        torch.cuda.synchronize()
        n = offsets[-1]
        close(replayed[0][:n], dx[0][:n], dx[1][:n], name="dx")
        for p in range(2):
            close(replayed[1 + p], dw[0][p], dw[1][p], name=f"dw{p}")
            close(replayed[3 + p], dw[0][p], dw[1][p], name=f"dw{p} alone")
        if offsets == [0, 2000, 2000, 2600]:
            assert all(torch.equal(a, b) for a, b in zip(first, replayed))
        here, there = outputs(), outputs()
        torch.cuda.synchronize()
        for _ in range(5):
            step(*here)
            with torch.cuda.stream(side):
                step(*there)
        torch.cuda.synchronize()
        assert all(torch.equal(a[:n] if a.shape[0] == R else a, b[:n] if b.shape[0] == R else b)
                   for got in (here, there) for a, b in zip(got, replayed))
    assert m.moe_check_status() == 0


# counts that end at, before and after every unit in which a kernel may take rows
@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 2])
def test_every_count_of_rows(P):
    counts = [0, 1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 0, 47, 48, 49, 63, 64, 65, 95, 96, 97, 127, 128, 129, 159, 160, 161, 191, 192,
              193, 223, 224, 225, 255, 256, 257, 0]
    off = np.concatenate([[0], np.cumsum(counts)])
    c = Case(int(off[-1]) + 11, 136, 200, len(counts), P, off)  # (and rows of no slot behind the last)
    y, dx, dw = c.reference()
    close(c.forward(), *y, name="y")
    got = c.backward()
    assert m.moe_check_status() == 0
    close(got[0], *dx, name="dx")
    for p in range(P):
        close(got[1][p], dw[0][p], dw[1][p], name=f"dw{p}")


# many rows a slot; with 48 slots so many tiles too that those of dw are twice as high, with heights that
# end in either half of one
@pytest.mark.gpu
@pytest.mark.parametrize("K,N,P,times", [(136, 200, 1, 1), (1288, 776, 2, 1), (264, 520, 2, 4), (520, 1032, 1, 4), (776, 264, 2, 4)])
def test_slots_of_many_rows(K, N, P, times):
    counts = [0, 1, 31, 300, 513, 1025, 0, 576, 97, 2000, 16, 250] * times
    off = np.concatenate([[0], np.cumsum(counts)])
    c = Case(int(off[-1]) + 5, K, N, len(counts), P, off, seed=12)
    y, dx, dw = c.reference()
    close(c.forward(), *y, name="y")
    got = c.backward()
    close(got[0], *dx, name="dx")
    for p in range(P):
        close(got[1][p], dw[0][p], dw[1][p], name=f"dw{p}")
    wide = c.backward(dx_type=F32, dw_type=F32)
    close(wide[0], *dx, name="dx fp32")
    added = c.backward(dx=False, dw_type=F32, add_dw=True, fill=1.0)
    for p in range(P):
        close(wide[1][p], dw[0][p], dw[1][p], name=f"dw{p} fp32")
        close(added[1][p], dw[0][p] + 1.0, dw[1][p] + STEP * (dw[0][p].abs() + 1.0), name=f"dw{p} added")
    assert m.moe_check_status() == 0
    # the first row of a slot is not its neighbour's, whatever it holds
    for r in (int(off[4]), int(off[5]), int(off[8]), int(off[10]), c.R - 1):
        c.x[r, 3], c.dy[r, 5] = float("inf"), float("nan")
    got = c.backward()
    for s in (1, 2, 3, 9, 11):
        close(got[1][0][s], dw[0][0][s], dw[1][0][s], name="dw beside infinities")


@pytest.mark.gpu
@pytest.mark.parametrize("K,N,P,times", [(144, 200, 2, 1), (784, 1032, 1, 1), (272, 520, 2, 8), (528, 1032, 1, 8), (784, 264, 2, 8)])
def test_weight_gradient_of_many_rows_kept_in_8_bits(K, N, P, times):
    counts = [700, 0, 1, 513, 1030, 97] if times == 1 else [170, 0, 1, 129, 64, 95] * times
    off = np.concatenate([[0], np.cumsum(counts)])
    c = Case(int(off[-1]) + 5, K, N, len(counts), P, off, seed=13)
    g = torch.Generator().manual_seed(K)
    # (codes and scales by themselves: every code is a value, the scale of a row any power of two)
    codes = torch.randint(0, 256, (c.R, K), generator=g).to(torch.uint8)
    codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes)
    scales = torch.exp2(torch.randint(-12, 4, (c.R, -(-K // 128)), generator=g).float())
    values = (codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)[:, :K]).to(BF)
    _, got = c.backward(dx=False, eight=(codes, scales))
    assert m.moe_check_status() == 0
    _, _, dw = c.reference(values)
    for p in range(P):
        close(got[p], dw[0][p], dw[1][p], name=f"dw{p}")


@pytest.mark.gpu
@pytest.mark.parametrize("R,K,N,S,P", [(100, 72, 136, 5, 2), (700, 600, 328, 3, 1), (45, 264, 512, 9, 2)])
def test_fp32_outputs_written_and_added(R, K, N, S, P):
    c = Case(R, K, N, S, P, seed=5)
    y, dx, dw = c.reference()
    got_y = c.forward(F32)
    close(got_y, *y, name="y")
    got = c.backward(dx_type=F32, dw_type=F32)
    close(got[0], *dx, name="dx")
    added = c.backward(dx_type=F32, dw_type=F32, add_dx=True, add_dw=True, fill=1.0)
    there = ~torch.isnan(dx[0])
    # (one more rounding, of the sum with what was there)
    close(added[0], torch.where(there, dx[0] + 1.0, 1.0), torch.where(there, dx[1] + STEP * (dx[0].abs() + 1.0), 0.0), name="dx added")
    for p in range(P):
        close(got[1][p], dw[0][p], dw[1][p], name=f"dw{p}")
        close(added[1][p], dw[0][p] + 1.0, dw[1][p] + STEP * (dw[0][p].abs() + 1.0), name=f"dw{p} added")
    out = torch.full((R, P * N), 2.0, device="cuda")
    c.forward(F32, add=True, out=out)
    there = ~torch.isnan(y[0])
    close(out, torch.where(there, y[0] + 2.0, 2.0), torch.where(there, y[1] + STEP * (y[0].abs() + 2.0), 0.0), name="y added")
    assert m.moe_check_status() == 0


def keep(x):
    """moe_checkpoint_rows by its definition: codes (as values), scales, in 64 bits, on the CPU."""
    R, C = x.shape
    nb = -(-C // 128)
    codes, scales = torch.zeros(R, C, dtype=torch.float64), torch.ones(R, nb, dtype=torch.float64)
    for b in range(nb):
        v = x[:, b * 128:(b + 1) * 128].double()
        for r in range(R):
            fine = v[r][torch.isfinite(v[r])].abs()
            top = float(fine.max()) if fine.numel() else 0.0
            e = 0
            if top:
                e = -117
                while top > 448.0 * 2.0 ** e and e < 119:
                    e += 1
            scales[r, b] = 2.0 ** e
        q = v / scales[:, b:b + 1]
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -300))).clamp(min=-6.0) - 3.0)
        codes[:, b * 128:(b + 1) * 128] = torch.where(torch.isfinite(v), (torch.round(q / step) * step).clamp(-448.0, 448.0), float("nan"))
    return codes, scales


def kept(x):
    """(uint8 codes, fp32 scales, the values they stand for in bf16)"""
    codes, scales = keep(x)
    values = codes * scales.repeat_interleave(128, 1)[:, :x.shape[1]]
    return codes.float().to(torch.float8_e4m3fn).view(torch.uint8), scales.float(), values.to(BF)


def same(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.gpu
@pytest.mark.parametrize("R,K,N,S,P", [(1, 16, 8, 1, 1), (17, 64, 128, 3, 2), (65, 144, 136, 5, 1), (300, 608, 328, 4, 2), (700, 272, 520, 2, 1),
                                       (333, 1040, 264, 40, 1)])
def test_weight_gradient_of_rows_kept_in_8_bits(R, K, N, S, P):
    c = Case(R, K, N, S, P, seed=9)
    c.x = (c.x.float() * torch.exp2(torch.randint(-6, 7, (R, K), generator=torch.Generator().manual_seed(R)).float())).to(BF)
    codes, scales, values = kept(c.x)
    for types in (BF, F32):
        _, got = c.backward(dx=False, eight=(codes, scales), dw_type=types)
        assert m.moe_check_status() == 0
        _, _, dw = c.reference(values)
        for p in range(P):
            close(got[p], dw[0][p], dw[1][p], name=f"dw{p}")


def rows_with_everything(R, C, seed=0):
    g = torch.Generator().manual_seed(seed + R * 1000 + C)
    x = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-12, 13, (R, C), generator=g).float())
    x = x * torch.exp2(torch.randint(-110, 100, (R, 1), generator=g).float()) if R > 2 else x
    x = x.to(BF)
    if R > 3:
        x[1] = 0.0
        x[2, ::3] = float("nan")
        x[2, 1::3] = float("inf")
        x[3, -1] = float("-inf")
    if R > 6:
        x[4] = 0.0
        x[4, -1] = 448.0 * 2.0 ** 20                   # the very border of a scale
        x[5] = x[5].sign() * 2.0 ** -133               # the smallest bf16
        x[6] = 3.3895e38                               # the largest
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("R,C", [(1, 8), (1, 128), (3, 136), (9, 600), (33, 264), (7, 1000), (500, 72), (40, 2048)])
def test_rows_kept_in_8_bits(R, C):
    x = rows_with_everything(R, C)
    codes = torch.full((R, C), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((R, -(-C // 128)), float("nan"), device="cuda")
    m.moe_checkpoint_rows(R, C, x.cuda(), codes, scale)
    want, scales = keep(x)
    assert torch.equal(scale.cpu().double(), scales)
    assert same(codes.cpu().view(torch.float8_e4m3fn).double(), want)
    # what is kept is a bf16 value
    values = want * scales.repeat_interleave(128, 1)[:, :C]
    assert same(values.to(BF).double(), values)


def swiglu_values(g, u):
    s = torch.sigmoid(g)
    return s, g * s * u


@pytest.mark.gpu
@pytest.mark.parametrize("R,I", [(1, 8), (8, 2048), (3, 136), (33, 328), (257, 264), (1000, 40)])
def test_swiglu_kept_in_8_bits_and_its_gradient(R, I):
    gen = torch.Generator().manual_seed(R + I)
    gu = (torch.randn(R, 2 * I, generator=gen) * torch.exp2(torch.randint(-6, 6, (R, 2 * I), generator=gen).float())).to(BF)
    gu[0, 0], gu[-1, 1], gu[0, 2] = -100.0, 100.0, -88.0  # saturated gates
    dh = torch.randn(R, I, generator=gen).to(BF)
    h = torch.full((R, I), float("nan"), dtype=BF, device="cuda")
    codes = torch.full((R, 2 * I), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((R, 2 * -(-I // 128)), float("nan"), device="cuda")
    m.moe_swiglu_checkpoint(R, I, gu.cuda(), h, codes, scale)
    kg, ku = keep(gu[:, :I]), keep(gu[:, I:])
    assert torch.equal(scale.cpu().double(), torch.cat([kg[1], ku[1]], 1))
    assert torch.equal(codes.cpu().view(torch.float8_e4m3fn).double(), torch.cat([kg[0], ku[0]], 1))

    def check(got, want, size, name):
        # size: the magnitude of the factors whose errors reach the value
        tol = HALF * (want.abs() + 2.0 ** -16 * size) + 2.0 ** -16 * size + 1e-30
        bad = ~((got.cpu().double() - want).abs() <= tol)
        assert not bool(bad.any()), (name, int(bad.sum()))

    want = swiglu_values(gu[:, :I].double(), gu[:, I:].double())[1]
    check(h, want, want.abs(), "h")
    g, u = (k[0] * k[1].repeat_interleave(128, 1)[:, :I] for k in (kg, ku))
    s, act = swiglu_values(g, u)
    d = dh.double()
    rest = torch.sigmoid(-g)
    for with_h in (True, False):
        out = torch.full((R, 2 * I), float("nan"), dtype=BF, device="cuda")
        again = torch.full((R, I), float("nan"), dtype=BF, device="cuda") if with_h else None
        m.moe_swiglu_backward(R, I, codes, scale, dh.cuda(), out, again)
        check(out[:, :I], d * u * s * (1.0 + g * rest), (d * u * s).abs() * (1.0 + (g * rest).abs()), "d_gate")
        check(out[:, I:], d * g * s, (d * g * s).abs(), "d_up")
        if with_h:
            check(again, act, act.abs(), "h again")
    assert m.moe_check_status() == 0


@pytest.mark.gpu
def test_swiglu_gradient_against_differences():
    """d/dg and d/du of sum(dh * h) at the kept values, by central differences in 64 bits."""
    R, I = 40, 64
    gen = torch.Generator().manual_seed(1)
    gu, dh = torch.randn(R, 2 * I, generator=gen).to(BF), torch.randn(R, I, generator=gen).to(BF)
    _, _, values = zip(kept(gu[:, :I]), kept(gu[:, I:]))
    g, u = (v.double() for v in values)
    codes, scale = torch.empty(R, 2 * I, dtype=torch.uint8, device="cuda"), torch.empty(R, 2, device="cuda")
    h, out = torch.empty(R, I, dtype=BF, device="cuda"), torch.empty(R, 2 * I, dtype=BF, device="cuda")
    m.moe_swiglu_checkpoint(R, I, gu.cuda(), h, codes, scale)
    m.moe_swiglu_backward(R, I, codes, scale, dh.cuda(), out)
    f = lambda a, b: dh.double() * swiglu_values(a, b)[1]  # noqa: E731
    e = 1e-5
    dg, du = (f(g + e, u) - f(g - e, u)) / (2 * e), (f(g, u + e) - f(g, u - e)) / (2 * e)
    got = out.cpu().double()
    # the differences are off by e^2 / 6 of the third derivative and 2^-52 / e of the value: under 1e-9
    for a, b in ((got[:, :I], dg), (got[:, I:], du)):
        assert bool(((a - b).abs() <= HALF * b.abs() + 1e-6).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 7168), (16, 2, 64), (100, 4, 600), (33, 3, 1000), (5, 32, 264), (300, 6, 2056), (64, 2, 9000)])
def test_combine_gradient(T, k, H):
    gen = torch.Generator().manual_seed(T + k + H)
    dout, y = torch.randn(T, H, generator=gen).to(BF), torch.randn(T * k, H, generator=gen).to(BF)
    w, perm = torch.rand(T, k, generator=gen), torch.randperm(T * k, generator=gen).int()
    shape = m.Shape(H, 8, 32, k, 0, 0, 32, 1)
    dy = torch.full((T * k, H), float("nan"), dtype=BF, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    m.moe_combine_backward(shape, T, dout.cuda(), y.cuda(), perm.cuda(), w.cuda(), dy, dw)
    assert m.moe_check_status() == 0
    row = perm.long()
    want = (w.double()[:, :, None] * dout.double()[:, None, :]).view(T * k, H)
    got = dy.cpu().double()[row]
    # (the product rounds to fp32 first)
    assert bool(((got - want).abs() <= (HALF + 2.0 ** -23) * want.abs() + 1e-40).all())
    terms = y.double()[row].view(T, k, H) * dout.double()[:, None, :]
    assert bool(((dw.cpu().double() - terms.sum(2)).abs() <= H * 2.0 ** -24 * terms.abs().sum(2) + 1e-30).all())


@pytest.mark.gpu
def test_a_row_that_combine_does_not_have():
    T, k, H = 6, 2, 64
    shape = m.Shape(H, 8, 4, k, 0, 0, 4, 1)
    dout, y, w = torch.ones(T, H, dtype=BF, device="cuda"), torch.ones(T * k, H, dtype=BF, device="cuda"), torch.ones(T, k, device="cuda")
    perm = torch.arange(T * k, dtype=torch.int32, device="cuda")
    perm[3], perm[7] = -1, T * k
    dy, dw = torch.full((T * k, H), 5.0, dtype=BF, device="cuda"), torch.full((T, k), 5.0, device="cuda")
    m.moe_combine_backward(shape, T, dout, y, perm, w, dy, dw)
    assert m.moe_check_status() == m.MOE_ERR_DEVICE_STATUS
    want = torch.full((T * k,), float(H))
    want[3] = want[7] = 0.0
    assert torch.equal(dw.cpu().view(-1), want)
    rows = torch.ones(T * k)
    rows[3] = rows[7] = 5.0
    assert torch.equal(dy.cpu().float()[:, 0], rows)


@pytest.mark.gpu
def test_offsets_that_do_not_fit_are_cut():
    """Offsets below zero, past the rows and backwards: the status is set, nothing outside is touched."""
    R, K, N, S = 50, 72, 136, 6
    c = Case(R, K, N, S, 1, [0, 10, 40, 30, 45, 60, 70], seed=2)
    cut = Case(R, K, N, S, 1, [0, 10, 40, 40, 45, 50, 50], seed=2)
    got = [c.forward(), *c.backward()]
    assert m.moe_check_status() == m.MOE_ERR_DEVICE_STATUS
    # slot 3 begins at its own offset, which slot 1 has passed: both have rows 30..39
    y, dx, dw = cut.reference()
    rows = torch.arange(R) >= 40
    rows[:30] = True
    close(got[0][rows.cuda()], y[0][rows], y[1][rows], name="y")
    close(got[1][rows.cuda()], dx[0][rows], dx[1][rows], name="dx")
    for s in (0, 1, 4):
        close(got[2][0][s], dw[0][0][s], dw[1][0][s], name="dw")
    assert bool((got[2][0][2] == 0).all()) and bool((got[2][0][5] == 0).all())
    neg = Case(R, K, N, S, 1, [-5, 10, 20, 20, 20, 20, 20], seed=2)
    fit = Case(R, K, N, S, 1, [0, 10, 20, 20, 20, 20, 20], seed=2)
    close(neg.forward(), *fit.reference()[0], name="y")
    assert m.moe_check_status() == m.MOE_ERR_DEVICE_STATUS


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_an_infinity_stays_in_its_row_and_slot(bad):
    """Rows of the next slot in a kernel's last chunk of a slot, and rows of no slot behind it."""
    off = [0, 37, 37, 101, 230]
    c = Case(240, 136, 264, 4, 2, off, seed=4)
    y, dx, dw = c.reference()
    clean = c.x.clone(), c.dy.clone()
    for r in (37, 101, 235):  # the first row of slots 2 and 3, and a row of no slot
        c.x[r, 5], c.dy[r, 7] = bad, bad
    gy, (gx, gw) = c.forward(), c.backward()
    assert m.moe_check_status() == 0
    hit = torch.zeros(240, dtype=torch.bool)
    hit[[37, 101]] = True
    assert not bool(torch.isfinite(gy.cpu()[hit]).any()) and not bool(torch.isfinite(gx.cpu()[hit]).any())
    close(gy[~hit.cuda()], y[0][~hit], y[1][~hit], name="y")
    close(gx[~hit.cuda()], dx[0][~hit], dx[1][~hit], name="dx")
    for p in range(2):
        for s in (0, 1):
            close(gw[p][s], dw[0][p][s], dw[1][p][s], name="dw")
        for s in (2, 3):
            w = gw[p][s].cpu()
            assert not bool(torch.isfinite(w[:, 5]).any())
            assert bool(torch.isfinite(w[[n for n in range(264) if p or n != 7]][:, [k for k in range(136) if k != 5]]).all())
    c.x, c.dy = clean


@pytest.mark.gpu
def test_nothing_but_the_outputs_is_written():
    """Guards around every output, and rows of no slot."""
    R, K, N, S, P = 130, 72, 136, 3, 2
    c = Case(R, K, N, S, P, [0, 33, 100, 117], seed=6)

    def guarded(n, dtype):
        t = torch.full((n + 4096,), 7.0, dtype=dtype, device="cuda")
        return t, t[2048:2048 + n]

    for dtype in (BF, F32):
        out, o = guarded(R * P * N, dtype)
        dx, d = guarded(R * K, dtype)
        dw, g = guarded(S * N * K, dtype)
        dw2, g2 = guarded(S * N * K, dtype)
        c.forward(dtype, out=o.view(R, P * N))
        w, w2 = c.weights()
        m.moe_expert_project_backward(c.p, R, c.dy.cuda(), c.x.cuda(), None, None, c.offsets(), w, w2, d.view(R, K), g.view(S, N, K),
                                      g2.view(S, N, K))
        assert m.moe_check_status() == 0
        for t in (out, dx, dw, dw2):
            assert bool((t[:2048] == 7.0).all()) and bool((t[-2048:] == 7.0).all())
        assert bool((o.view(R, -1)[117:] == 7.0).all()) and bool((d.view(R, -1)[117:] == 7.0).all())


@pytest.mark.gpu
def test_one_gradient_at_a_time_no_rows_and_repeats():
    c = Case(150, 264, 136, 4, 2, seed=8)
    dx, dw = c.backward()
    assert torch.equal(c.backward(dw=False)[0][:c.off[-1]], dx[:c.off[-1]])
    only = c.backward(dx=False)[1]
    for a, b in zip(only, dw):
        assert torch.equal(a, b)
    first, again = c.forward(), c.forward()
    assert torch.equal(first.nan_to_num(9.0), again.nan_to_num(9.0))
    none = torch.full((4, 136, 264), 3.0, dtype=BF, device="cuda")
    w, w2 = c.weights()
    empty = torch.empty(0, 264, dtype=BF, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    m.moe_expert_project_backward(c.p, 0, empty.new_empty(0, 272), empty, None, None, off, w, w2, empty, none, none.clone())
    torch.cuda.synchronize()
    assert bool((none == 0).all())
    held = torch.full((4, 136, 264), 3.0, device="cuda")
    m.moe_expert_project_backward(c.p, 0, empty.new_empty(0, 272), empty, None, None, off, w, w2, empty, held, held.clone(), add_dw=True)
    torch.cuda.synchronize()
    assert bool((held == 3.0).all())
    m.moe_expert_project(c.p, 0, empty, off, w, w2, empty.new_empty(0, 272))
    # all slots empty, with rows: dw is zero, no row is written
    c.off[:] = 0
    dx, dw = c.backward()
    assert m.moe_check_status() == 0
    assert bool(torch.isnan(dx).all()) and all(bool((g == 0).all()) for g in dw)


@pytest.mark.gpu
def test_captured_in_a_graph_and_on_another_stream():
    c = Case(300, 264, 136, 4, 2, seed=10)
    want_y, (want_dx, want_dw) = c.forward(), c.backward()
    n = int(c.off[-1])
    x, dy, off, (w, w2) = c.x.cuda(), c.dy.cuda(), c.offsets(), c.weights()
    out = torch.zeros(300, 272, dtype=BF, device="cuda")
    dx, dw, dw2 = torch.zeros(300, 264, dtype=BF, device="cuda"), torch.zeros_like(w), torch.zeros_like(w)
    codes, scale = torch.empty(300, 264, dtype=torch.uint8, device="cuda"), torch.empty(300, 3, device="cuda")
    act, gu, dgu = (torch.zeros(300, i, dtype=BF, device="cuda") for i in (136, 272, 272))
    kept_gu, kept_scale = torch.empty(300, 272, dtype=torch.uint8, device="cuda"), torch.empty(300, 4, device="cuda")

    def step():
        m.moe_expert_project(c.p, 300, x, off, w, w2, out)
        m.moe_swiglu_checkpoint(300, 136, out, act, kept_gu, kept_scale)
        m.moe_checkpoint_rows(300, 264, x, codes, scale)
        m.moe_expert_project_backward(c.p, 300, dy, x, None, None, off, w, w2, dx, dw, dw2)
        m.moe_swiglu_backward(300, 136, kept_gu, kept_scale, act, dgu)

    step()
    torch.cuda.synchronize()
    plain = [t.clone() for t in (out, dx, dw, dw2, act, codes, scale, dgu)]
    assert torch.equal(out[:n], want_y[:n]) and torch.equal(dx[:n], want_dx[:n]) and torch.equal(dw, want_dw[0])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in (out, dx, dw, dw2, act, dgu):
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(plain, (out, dx, dw, dw2, act, codes, scale, dgu)))
    for t in (out, dx, dw, dw2, act, dgu):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(plain, (out, dx, dw, dw2, act, codes, scale, dgu)))
    assert m.moe_check_status() == 0


@pytest.mark.gpu
def test_several_threads_and_streams_at_once():
    """Four host threads on streams of their own, different problems, no buffer shared: the results are those of calls alone."""
    import threading

    cases = [Case(300, 264, 136, 4, 2, seed=20), Case(60, 2056, 264, 2, 1, seed=21), Case(900, 136, 520, 40, 1, seed=22),
             Case(5, 72, 4104, 3, 2, seed=23)]
    want = [(c.forward().nan_to_num(9.0), *[t.nan_to_num(9.0) for t in (lambda g: [g[0], *g[1]])(c.backward())]) for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * len(cases), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(6):
                    y, (dx, dw) = cases[i].forward(), cases[i].backward()
                torch.cuda.current_stream().synchronize()
                got[i] = [t.nan_to_num(9.0) for t in (y, dx, *dw)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # reported below, in the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert m.moe_check_status() == 0
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def rows_close(got, want, tol):
    """The same as close() on the device."""
    tol = tol + HALF * (want.abs() + tol) + 1e-30
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.gpu
def test_outputs_of_more_than_2_31_elements():
    """y, dx and dw past 32-bit offsets: the first, a middle and the last rows and slots."""
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    S, K, N, P = 5, 72, 2048, 2
    R = 2 ** 31 // (P * N) + 1003
    off = torch.tensor([0, 17, 17, R // 2 + 5, R - 9, R - 2], dtype=torch.int32, device="cuda")
    x, w = new(R, K), [new(S, N, K) for _ in range(P)]
    y = torch.empty(R, P * N, dtype=BF, device="cuda")
    m.moe_expert_project(m.Project(K, N, S, P), R, x, off, *w, y)
    assert m.moe_check_status() == 0
    for s, rows in ((0, slice(0, 17)), (2, slice(R // 2 - 60, R // 2 + 5)), (4, slice(R - 9, R - 2))):
        for p in range(P):
            want = x[rows].double() @ w[p][s].double().t()
            rows_close(y[rows, p * N:(p + 1) * N], want, K * STEP * (x[rows].double().abs() @ w[p][s].double().abs().t()))
    # dx, as wide as y was: one part, its contraction short
    dx, dy = y, x[:, :64].contiguous()
    w = new(S, 64, P * N)
    m.moe_expert_project_backward(m.Project(P * N, 64, S), R, dy, None, None, None, off, w, None, dx, None)
    assert m.moe_check_status() == 0
    for s, rows in ((0, slice(0, 17)), (3, slice(R - 80, R - 9)), (4, slice(R - 9, R - 2))):
        rows_close(dx[rows], dy[rows].double() @ w[s].double(), 64 * STEP * (dy[rows].double().abs() @ w[s].double().abs()))
    del y, dx, x, dy, w
    S, K, N, R = 1024, 1032, 2064, 3000
    off = torch.linspace(0, R, S + 1, device="cuda").round().to(torch.int32)
    x, dy, dw = new(R, K), new(R, N), torch.empty(S, N, K, dtype=BF, device="cuda")
    m.moe_expert_project_backward(m.Project(K, N, S), R, dy, x, None, None, off, None, None, None, dw)
    assert m.moe_check_status() == 0
    for s in (0, 511, 1007, 1008, 1023):
        rows = slice(int(off[s]), int(off[s + 1]))
        a, b = dy[rows].double(), x[rows].double()
        rows_close(dw[s], a.t() @ b, len(a) * STEP * (a.abs().t() @ b.abs()))


@pytest.mark.gpu
def test_kept_rows_and_combine_of_more_than_2_31_elements():
    g = torch.Generator(device="cuda").manual_seed(2)
    H, k = 4096, 2
    n = 2 ** 31 // H + 250
    x = torch.randn(n, H, generator=g, device="cuda", dtype=BF)
    codes, scale = torch.empty(n, H, dtype=torch.uint8, device="cuda"), torch.empty(n, H // 128, device="cuda")
    m.moe_checkpoint_rows(n, H, x, codes, scale)
    for rows in (slice(0, 3), slice(n // 2, n // 2 + 3), slice(n - 3, n)):
        c, s = keep(x[rows].cpu())
        assert torch.equal(scale[rows].cpu().double(), s) and torch.equal(codes[rows].cpu().view(torch.float8_e4m3fn).double(), c)
    # the same memory as gate and up of 2048, and as what two experts gave each token
    I = H // 2
    h, dh = torch.empty(n, I, dtype=BF, device="cuda"), torch.randn(n, I, generator=g, device="cuda", dtype=BF)
    m.moe_swiglu_checkpoint(n, I, x, h, codes, scale)
    out, again = torch.empty_like(x), torch.empty_like(h)
    m.moe_swiglu_backward(n, I, codes, scale, dh, out, again)
    for rows in (slice(0, 3), slice(n - 3, n)):
        gate, up = (kept(v)[2].double() for v in (x[rows, :I].cpu(), x[rows, I:].cpu()))
        s, act = swiglu_values(gate, up)
        d, bound = dh[rows].cpu().double(), 2.0 ** -15
        assert bool(((again[rows].cpu().double() - act).abs() <= (HALF + bound) * act.abs() + 1e-30).all())
        want = d * gate * s
        assert bool(((out[rows, I:].cpu().double() - want).abs() <= (HALF + bound) * want.abs() + 1e-30).all())
    T = n // k
    shape = m.Shape(H, 8, 8, k, 0, 0, 8, 1)
    dout, w = torch.randn(T, H, generator=g, device="cuda", dtype=BF), torch.rand(T, k, generator=g, device="cuda")
    perm, dw = torch.randperm(T * k, generator=g, device="cuda").int(), torch.empty(T, k, device="cuda")
    x = x[:T * k]
    out = out[:T * k]
    m.moe_combine_backward(shape, T, dout, x, perm, w, out, dw)
    assert m.moe_check_status() == 0
    for t in (0, T // 2, T - 1):
        for j in range(k):
            row = int(perm[t * k + j])
            want = w[t, j].double() * dout[t].double()
            assert bool(((out[row].double() - want).abs() <= (HALF + 2.0 ** -23) * want.abs() + 1e-40).all())
            terms = dout[t].double() * x[row].double()
            assert abs(float(dw[t, j]) - float(terms.sum())) <= H * 2.0 ** -24 * float(terms.abs().sum())
    row = int((perm == T * k - 1).nonzero()[0])  # the very last row of y
    want = w.view(-1)[row].double() * dout[row // k].double()
    assert bool(((out[-1].double() - want).abs() <= (HALF + 2.0 ** -23) * want.abs() + 1e-40).all())


# ------------------------------------------------------------------ refusals (no GPU needed)
def project(p, rows=4, x=FAKE, off=FAKE, w=FAKE, w2=None, out=FAKE, kind=0):
    return m.lib().moe_expert_project(ctypes.byref(p) if p else None, rows, x, off, w, w2, out, kind, None)


def backward(p, rows=4, dy=FAKE, x=FAKE, x8=None, sc=None, off=FAKE, w=FAKE, w2=None, dx=FAKE, dxt=0, dw=FAKE, dw2=None, dwt=0):
    return m.lib().moe_expert_project_backward(ctypes.byref(p) if p else None, rows, dy, x, x8, sc, off, w, w2, dx, dxt, dw, dw2, dwt,
                                               None)


@pytest.mark.parametrize("p,code", [
    (None, m.MOE_ERR_INVALID_ARG), (m.Project(0, 8, 1), m.MOE_ERR_INVALID_ARG), (m.Project(8, -8, 1), m.MOE_ERR_INVALID_ARG),
    (m.Project(8, 8, 0), m.MOE_ERR_INVALID_ARG), (m.Project(12, 8, 1), m.MOE_ERR_INVALID_ARG), (m.Project(8, 20, 1), m.MOE_ERR_INVALID_ARG),
    (m.Project(8, 8, 1, 3), m.MOE_ERR_INVALID_ARG), (m.Project(8, 8, 1, 0), m.MOE_ERR_INVALID_ARG),
    (m.Project(8, 8, 1025), m.MOE_ERR_UNSUPPORTED), (m.Project((1 << 24) + 8, 8, 1), m.MOE_ERR_UNSUPPORTED),
    (m.Project(8, (1 << 24) + 8, 1), m.MOE_ERR_UNSUPPORTED)])
def test_sizes_are_refused(p, code):
    assert project(p) == code and m.last_error()
    assert backward(p) == code


def test_project_arguments_are_refused():
    p, two = m.Project(64, 64, 4), m.Project(64, 64, 4, 2)
    bad = m.MOE_ERR_INVALID_ARG
    assert project(p, rows=-1) == bad
    assert project(p, rows=2 ** 30) == m.MOE_ERR_UNSUPPORTED
    assert project(p, kind=3) == bad and project(p, kind=-1) == bad
    for name in ("x", "off", "w", "out"):
        assert project(p, **{name: None}) == bad
        assert project(p, **{name: FAKE + 2}) == bad
    assert project(two) == bad and "w2" in m.last_error()
    assert project(p, w2=FAKE) == bad and "n_parts" in m.last_error()
    assert project(p, rows=0, x=None, off=None, w=None, out=None) == m.MOE_OK


def test_backward_arguments_are_refused():
    p, two, narrow = m.Project(64, 64, 4), m.Project(64, 64, 4, 2), m.Project(72, 64, 4)
    bad = m.MOE_ERR_INVALID_ARG
    assert backward(p, rows=-1) == bad
    assert backward(p, dxt=3) == bad and backward(p, dwt=-1) == bad
    for name in ("dy", "off", "w", "x"):
        assert backward(p, **{name: None}) == bad
    for name in ("dy", "off", "w", "x", "dx", "dw"):
        assert backward(p, **{name: FAKE + 2}) == bad
    assert backward(two, w2=FAKE) == bad and "dw2" in m.last_error()
    assert backward(two, dw2=FAKE) == bad and "w2" in m.last_error()
    assert backward(p, dw2=FAKE) == bad and backward(p, dw=None, dw2=FAKE) == bad
    assert backward(p, x8=FAKE, sc=FAKE) == bad and "not both" in m.last_error()
    assert backward(p, x=None, x8=FAKE) == bad and "x8_scale" in m.last_error()
    assert backward(narrow, x=None, x8=FAKE, sc=FAKE) == bad and "16" in m.last_error()
    assert backward(p, dx=None, dw=None) == m.MOE_OK


def test_kept_rows_arguments_are_refused():
    lib, bad = m.lib(), m.MOE_ERR_INVALID_ARG
    for rows, cols in ((-1, 8), (4, 0), (4, -8), (4, 12)):
        assert lib.moe_checkpoint_rows(rows, cols, FAKE, FAKE, FAKE, None) == bad
        assert lib.moe_swiglu_checkpoint(rows, cols, FAKE, FAKE, FAKE, FAKE, None) == bad
        assert lib.moe_swiglu_backward(rows, cols, FAKE, FAKE, FAKE, FAKE, FAKE, None) == bad
    assert lib.moe_checkpoint_rows(4, 1 << 25, FAKE, FAKE, FAKE, None) == m.MOE_ERR_UNSUPPORTED
    assert lib.moe_checkpoint_rows(2 ** 31 - 1, 1 << 20, FAKE, FAKE, FAKE, None) == m.MOE_ERR_UNSUPPORTED
    for i in range(3):
        for wrong in (None, FAKE + 2):
            args = [FAKE] * 3
            args[i] = wrong
            assert lib.moe_checkpoint_rows(4, 8, *args, None) == bad
    for i in range(4):
        args = [FAKE] * 4
        args[i] = None
        assert lib.moe_swiglu_checkpoint(4, 8, *args, None) == bad
        assert lib.moe_swiglu_backward(4, 8, *args, FAKE, None) == bad
    assert lib.moe_swiglu_backward(4, 8, FAKE, FAKE, FAKE, FAKE, FAKE + 8, None) == bad
    assert lib.moe_checkpoint_rows(0, 8, None, None, None, None) == m.MOE_OK
    assert lib.moe_swiglu_checkpoint(0, 8, None, None, None, None, None) == m.MOE_OK
    assert lib.moe_swiglu_backward(0, 8, None, None, None, None, None, None) == m.MOE_OK


def test_combine_gradient_arguments_are_refused():
    lib, shape = m.lib(), ctypes.byref(m.Shape(64, 8, 8, 2, 0, 0, 8, 1))
    for i in range(6):
        for wrong in (None, FAKE + 2):
            args = [FAKE] * 6
            args[i] = wrong
            assert lib.moe_combine_backward(shape, 4, *args, None) == m.MOE_ERR_INVALID_ARG
    assert lib.moe_combine_backward(None, 4, *([FAKE] * 6), None) == m.MOE_ERR_INVALID_ARG
    assert lib.moe_combine_backward(shape, -1, *([FAKE] * 6), None) == m.MOE_ERR_INVALID_ARG
    assert lib.moe_combine_backward(shape, 0, *([None] * 6), None) == m.MOE_OK


def test_binding_refuses_other_sizes_and_types():
    p = m.Project(64, 32, 4, 2)
    bf = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    off, w = torch.zeros(5, dtype=torch.int32), bf(4, 32, 64)
    with pytest.raises(ValueError):
        m.moe_expert_project(p, 3, bf(3, 32), off, w, w, bf(3, 64))
    with pytest.raises(ValueError):  # the host's memory
        m.moe_expert_project(p, 3, bf(3, 64), off, w, w, bf(3, 64))
    with pytest.raises(ValueError):
        m.moe_expert_project(p, 3, None, off, None, None, bf(3, 64), add=True)
    with pytest.raises(ValueError):
        m.moe_expert_project(p, 3, None, off[:4], None, None, None)
    with pytest.raises(ValueError):  # both weight gradients are of one type
        m.moe_expert_project_backward(p, 3, None, None, None, None, None, None, None, None, w, w.float())
    with pytest.raises(ValueError):
        m.moe_checkpoint_rows(3, 136, None, None, torch.zeros(3, 1))
    with pytest.raises(ValueError):
        m.moe_swiglu_backward(3, 136, None, torch.zeros(3, 2), None, None)
