"""moe_swiglu_checkpoint and moe_swiglu_backward where gate, up or dh hold infinities, NaN and the type's extremes.

Tolerance, as in test_expert_training.py: one rounding to bf16 (half a step, 2^-8 of the value) and 2^-16 of the factors
that are rounded before.  The sigmoid is 1 / (1 + 2^(-g log2 e)): the product is rounded once and log2 e before it, both
2^-24 of up to 70 * 1.45 (beyond |g| = 70 the 1e-30 below covers what is left), 2 * 102 * 2^-24 * ln 2 = 71 steps of
2^-23; ex2.approx adds 2 of them, the sum half of one, rcp.approx one, the products beside it less than 10: 2^-16 is
128.  A sigmoid below 2^-126 counts as 0."""
import pytest
import torch

import moe_expert_layer_06_gb300 as m
from test_expert_training import BF, HALF, keep, same

INF, NAN, TOP = float("inf"), float("nan"), 3.3895e38


def sigmoid(g):
    s = torch.sigmoid(g)
    return torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)


def check(got, want, size, name):
    """Infinities and NaN in the same places; past bf16's range an infinity."""
    got = got.cpu().double()
    want = torch.where(want.abs() > 3.396e38, want.sign() * INF, want)
    there = torch.isfinite(want)
    assert same(got[~there], want[~there]), (name, got[~there], want[~there])
    tol = HALF * (want.abs() + 2.0 ** -16 * size) + 2.0 ** -16 * size + 1e-30
    bad = there & ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (name, bad.nonzero()[:4], got[bad][:4], want[bad][:4])


def run(gu, dh):
    R, I = dh.shape
    h, again = (torch.full((R, I), 7.0, dtype=BF, device="cuda") for _ in range(2))
    codes = torch.full((R, 2 * I), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((R, 2 * -(-I // 128)), 5.0, device="cuda")
    d = torch.full((R, 2 * I), 7.0, dtype=BF, device="cuda")
    m.moe_swiglu_checkpoint(R, I, gu.cuda(), h, codes, scale)
    m.moe_swiglu_backward(R, I, codes, scale, dh.cuda(), d, again)
    assert m.moe_check_status() == 0
    return h, codes, scale, d, again


@pytest.mark.gpu
@pytest.mark.parametrize("I", [8, 136, 256, 264, 520])
def test_infinities_and_nan_of_either_half(I):
    """Row by row: in the gate only, in the up only, in both, in a whole block of one, in whole rows, in dh."""
    R = 12
    gen = torch.Generator().manual_seed(I)
    gu, dh = torch.randn(R, 2 * I, generator=gen), torch.randn(R, I, generator=gen)
    gate, up = gu[:, :I], gu[:, I:]
    last = slice(I - min(I, 128 if I % 128 == 0 else I % 128), I)  # the last block
    for i, v in enumerate((INF, -INF, NAN)):
        gate[0, i], up[1, i] = v, v
        gate[2, i], up[2, -1 - i] = v, v
        dh[10, i] = v
    gate[3, last], up[4, last] = INF, NAN
    gate[5, last], up[5, last] = -INF, INF
    gate[6], up[7] = NAN, -INF
    gate[8], up[8] = INF, INF
    gate[9, 0], up[9, 1] = TOP, -TOP      # the largest, beside which the rest of the block is kept as 0
    gate[11], up[11] = -200.0, 1.0        # a sigmoid that counts as 0
    gu, dh = gu.to(BF), dh.to(BF)
    gate, up = gu[:, :I], gu[:, I:]
    h, codes, scale, d, again = run(gu, dh)
    kg, ku = keep(gate), keep(up)
    assert torch.equal(scale.cpu().double(), torch.cat([kg[1], ku[1]], 1))
    assert same(codes.cpu().view(torch.float8_e4m3fn).double(), torch.cat([kg[0], ku[0]], 1))
    g, u = gate.double(), up.double()
    want = g * sigmoid(g) * u
    check(h, want, want.abs(), "h")
    # the gradient is that of the kept values, in which an infinity is a NaN
    g, u = (k[0] * k[1].repeat_interleave(128, 1)[:, :I] for k in (kg, ku))
    s, rest, dd = sigmoid(g), torch.sigmoid(-g), dh.double()
    check(d[:, :I], dd * u * s * (1.0 + g * rest), (dd * u * s).abs() * (1.0 + (g * rest).abs()), "d_gate")
    check(d[:, I:], dd * g * s, (dd * g * s).abs(), "d_up")
    check(again, g * s * u, (g * s * u).abs(), "h again")


@pytest.mark.gpu
def test_gates_over_the_whole_range():
    """Every finite bf16 up to 2^7 as a gate (beyond, the sigmoid is 0 or 1 in fp64 too), whatever the sign."""
    bits = torch.arange(0x4300, dtype=torch.int32)
    gate = torch.cat([bits, bits | 0x8000]).to(torch.int16).view(BF).view(-1, 8)
    R = gate.shape[0]
    gen = torch.Generator().manual_seed(9)
    up, dh = torch.randn(R, 8, generator=gen).to(BF), torch.randn(R, 8, generator=gen).to(BF)
    h, codes, scale, d, again = run(torch.cat([gate, up], 1), dh)
    g, u = gate.double(), up.double()
    want = g * sigmoid(g) * u
    check(h, want, want.abs(), "h")
    kg, ku = keep(gate), keep(up)
    assert torch.equal(scale.cpu().double(), torch.cat([kg[1], ku[1]], 1))
    g, u = kg[0] * kg[1], ku[0] * ku[1]
    s, rest, dd = sigmoid(g), torch.sigmoid(-g), dh.double()
    check(d[:, :8], dd * u * s * (1.0 + g * rest), (dd * u * s).abs() * (1.0 + (g * rest).abs()), "d_gate")
    check(d[:, 8:], dd * g * s, (dd * g * s).abs(), "d_up")
    check(again, g * s * u, (g * s * u).abs(), "h again")


def keep_wide(x):
    """keep() of finite rows, vectorised: the least power of two (from 2^-117 on) that brings a block to 448 at most."""
    R, C = x.shape
    nb = -(-C // 128)
    v = torch.nn.functional.pad(x.double(), (0, nb * 128 - C)).view(R, nb, 128)
    frac, e = torch.frexp(v.abs().amax(2))  # (448 is 0.875 * 2^9)
    e = torch.where(frac == 0.0, 0, (e - 9 + (frac > 0.875).int()).clamp(min=-117))
    scale = torch.ldexp(torch.ones_like(frac), e)
    q = v / scale[:, :, None]
    step = torch.ldexp(torch.ones_like(q), (torch.frexp(q)[1] - 1).clamp(min=-6) - 3)
    return (torch.round(q / step) * step).view(R, nb * 128)[:, :C], scale


@pytest.mark.gpu
@pytest.mark.parametrize("C", [128 * 4095, 128 * 4095 + 8, 128 * 4096, 128 * 4096 + 8, 128 * 9001 + 72])
def test_rows_of_many_blocks(C):
    """Around 4096 blocks a row, where a block's row is found in another way."""
    R = 3
    gen = torch.Generator().manual_seed(C)
    x = (torch.randn(R, C, generator=gen) * torch.exp2(torch.randint(-9, 10, (R, 1), generator=gen).float())).to(BF)
    want, scales = keep_wide(x)
    assert torch.equal(keep(x[:, -200:])[1], keep_wide(x[:, -200:])[1]) and torch.equal(keep(x[:, -200:])[0], keep_wide(x[:, -200:])[0])
    codes, scale = torch.full((R, C), 0x55, dtype=torch.uint8, device="cuda"), torch.full(scales.shape, 5.0, device="cuda")
    m.moe_checkpoint_rows(R, C, x.cuda(), codes, scale)
    assert torch.equal(scale.cpu().double(), scales) and torch.equal(codes.cpu().view(torch.float8_e4m3fn).double(), want)
    up, dh = torch.randn(R, C, generator=gen).to(BF), torch.randn(R, C, generator=gen).to(BF)
    h, codes, scale, d, again = run(torch.cat([x, up], 1), dh)
    ku = keep_wide(up)
    assert torch.equal(scale.cpu().double(), torch.cat([scales, ku[1]], 1))
    assert torch.equal(codes.cpu().view(torch.float8_e4m3fn).double(), torch.cat([want, ku[0]], 1))
    g, u = x.double(), up.double()
    check(h, g * sigmoid(g) * u, (g * sigmoid(g) * u).abs(), "h")
    g, u = (k[0] * k[1].repeat_interleave(128, 1)[:, :C] for k in ((want, scales), ku))
    s, rest, dd = sigmoid(g), torch.sigmoid(-g), dh.double()
    check(d[:, :C], dd * u * s * (1.0 + g * rest), (dd * u * s).abs() * (1.0 + (g * rest).abs()), "d_gate")
    check(d[:, C:], dd * g * s, (dd * g * s).abs(), "d_up")
    check(again, g * s * u, (g * s * u).abs(), "h again")
