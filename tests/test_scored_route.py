"""Scored routing and its gradient (moe_route_scored, moe_route_scored_backward)
against their definition in 64 bits.

Tolerances.  A weight is exp of a difference of logits (its argument is off by
half a step of at most A = max |logit|, so the value by A * 2^-24 relative; expf
itself by 2 steps), a sum of k of them, a quotient and a product: (A + k + 16)
roundings of 2^-24 relative cover them.  A gradient is a product of up to four
such values with (g - sum w g), each at most max |g| * scale: 4 (A + k + 16)
roundings of that size.  The dense softmax adds a sum over E values in a tree
of lanes (E / 32 + 5 steps deep)."""
import ctypes

import numpy as np
import pytest
import torch

import moe_expert_layer_06_gb300 as m
import moe_inputs as mi

INF = float("inf")
FAKE = 0x10000  # aligned address that is never dereferenced on the host


def shape_of(E, k, hidden=8):
    return m.Shape(hidden, 8, E, k, 0, 0, E, 1)


def reference(l, bias, r, k):
    """(idx, w, s, kept) by the definition, fp64 on the CPU."""
    l = l.double().cpu()
    T, E = l.shape
    l = torch.where(torch.isnan(l), torch.full_like(l, -INF), l)
    masked = l == -INF
    if r.score == m.MOE_SCORE_SIGMOID:
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(1, keepdim=True)
        s = torch.where(l == top, torch.ones_like(l), torch.exp(l - top))
        s = torch.where(masked, torch.zeros_like(l), s)
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    c = s + (bias.double().cpu() if bias is not None else 0.0)
    c = c.masked_fill(masked, -INF).numpy()
    gs = E // r.n_groups
    idx = np.zeros((T, k), dtype=np.int64)
    for t in range(T):
        allowed = list(range(r.n_groups))
        if r.topk_groups < r.n_groups:
            g = []
            for i in range(r.n_groups):
                b = sorted(c[t, i * gs:(i + 1) * gs], reverse=True)
                g.append(b[0] + (b[1] if r.group_score == m.MOE_GROUP_TOP2 and gs > 1 and b[1] > -INF else 0.0))
            allowed = sorted(range(r.n_groups), key=lambda i: (-g[i], i))[:r.topk_groups]
        pool = [e for i in allowed for e in range(i * gs, (i + 1) * gs)]
        idx[t] = sorted(pool, key=lambda e: (-c[t, e], e))[:k]
    idx = torch.from_numpy(idx)
    lk, sk = l.gather(1, idx), s.gather(1, idx)
    if r.renormalize:
        low = lk.clamp(max=0.0) if r.score == m.MOE_SCORE_SIGMOID else lk
        top = low.amax(1, keepdim=True)
        e = torch.where(low == top, torch.ones_like(low), torch.exp(low - top))
        if r.score == m.MOE_SCORE_SIGMOID:
            e = e / (1.0 + torch.exp(-lk.abs()))
        e = torch.where(lk == -INF, torch.zeros_like(e), e)
        w = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = sk
    return idx, w * r.scale, s, l


def reference_grad(l, idx, s, w, g, r):
    """d logits by the formulas, fp64."""
    g = g.double().cpu()
    lk = l.gather(1, idx)
    rest = 1.0 / (1.0 + torch.exp(lk))
    d = torch.zeros_like(l)
    if r.renormalize:
        u = w / r.scale
        v = r.scale * u * (g - (u * g).sum(1, keepdim=True))
        d.scatter_(1, idx, v * rest if r.score == m.MOE_SCORE_SIGMOID else v)
    elif r.score == m.MOE_SCORE_SIGMOID:
        d.scatter_(1, idx, r.scale * g * s.gather(1, idx) * rest)
    else:
        ds = torch.zeros_like(l).scatter_(1, idx, r.scale * g)
        d = s * (ds - (ds * s).sum(1, keepdim=True))
    return torch.where(l == -INF, torch.zeros_like(d), d)


def call(l, bias, r, k, logits_out=None):
    T, E = l.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    m.moe_route_scored(shape_of(E, k), r, T, None, None, bias, l, logits_out, idx, w)
    assert m.moe_check_status() == 0
    return idx, w


def check(l, bias, r, k, seed=0):
    T, E = l.shape
    idx, w = call(l, bias, r, k)
    ridx, rw, s, lm = reference(l, bias, r, k)
    assert torch.equal(idx.cpu().long(), ridx)
    A = float(lm[lm.abs() < 1e30].abs().max()) if bool((lm.abs() < 1e30).any()) else 0.0
    steps = A + k + 16 + (E / 32 + 5 if r.score == m.MOE_SCORE_SOFTMAX else 0)
    err = (w.double().cpu() - rw).abs()
    assert bool((err <= steps * 2.0 ** -24 * rw.abs() + 1e-37).all()), float((err / rw.abs().clamp(min=1e-30)).max())
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(seed))
    d = torch.full((T, E), float("nan"), device="cuda")
    m.moe_route_scored_backward(shape_of(E, k), r, T, l, idx, g.cuda(), d)
    assert m.moe_check_status() == 0
    want = reference_grad(lm, ridx, s, rw, g, r)
    tol = 4 * steps * 2.0 ** -24 * abs(r.scale) * g.double().abs().amax(1, keepdim=True)
    assert bool(((d.double().cpu() - want).abs() <= tol).all())


ROUTERS = [
    (256, 8, m.Router(m.MOE_SCORE_SIGMOID, 8, 4, m.MOE_GROUP_TOP2, 1, 2.5)),
    (256, 8, m.Router(m.MOE_SCORE_SOFTMAX, 1, 1, m.MOE_GROUP_MAX, 0, 1.0)),
    (256, 8, m.Router(m.MOE_SCORE_SOFTMAX, 8, 3, m.MOE_GROUP_MAX, 1, 1.0)),
    (64, 6, m.Router(m.MOE_SCORE_SIGMOID, 1, 1, m.MOE_GROUP_MAX, 0, 1.5)),
    (60, 4, m.Router(m.MOE_SCORE_SOFTMAX, 1, 1, m.MOE_GROUP_MAX, 1, 1.0)),
    (72, 6, m.Router(m.MOE_SCORE_SIGMOID, 8, 2, m.MOE_GROUP_TOP2, 1, 1.0)),   # groups of 9
    (160, 6, m.Router(m.MOE_SCORE_SOFTMAX, 8, 3, m.MOE_GROUP_TOP2, 0, 16.0)),  # groups of 20
    (8, 2, m.Router(m.MOE_SCORE_SOFTMAX, 1, 1, m.MOE_GROUP_MAX, 1, 1.0)),
    (1, 1, m.Router(m.MOE_SCORE_SIGMOID, 1, 1, m.MOE_GROUP_TOP2, 1, 1.0)),
    (32, 32, m.Router(m.MOE_SCORE_SIGMOID, 32, 32, m.MOE_GROUP_TOP2, 1, 1.0)),  # every expert
    (64, 4, m.Router(m.MOE_SCORE_SIGMOID, 32, 5, m.MOE_GROUP_TOP2, 0, 1.0)),  # groups of 2
    (512, 10, m.Router(m.MOE_SCORE_SIGMOID, 16, 5, m.MOE_GROUP_TOP2, 1, 2.5)),
    (1000, 7, m.Router(m.MOE_SCORE_SOFTMAX, 4, 3, m.MOE_GROUP_MAX, 0, 1.0)),
    (1024, 32, m.Router(m.MOE_SCORE_SIGMOID, 1, 1, m.MOE_GROUP_MAX, 1, 1.0)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 65, 1001])
@pytest.mark.parametrize("E,k,r", ROUTERS)
@pytest.mark.parametrize("biased", [False, True])
def test_matches_the_definition(E, k, r, T, biased):
    g = torch.Generator().manual_seed(E + 7 * T + k)
    l = (torch.randn(T, E, generator=g) * 1.7).cuda()
    bias = (torch.randn(E, generator=g) * 0.1).cuda() if biased else None
    check(l, bias, r, k, T)


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,r", ROUTERS)
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lower_expert(E, k, r, biased):
    """Few distinct logits (and biases): most comparisons are ties."""
    g = torch.Generator().manual_seed(E)
    l = torch.randint(-2, 3, (65, E), generator=g).float().cuda()
    l[0] = 0.0
    bias = (torch.randint(0, 2, (E,), generator=g).float() * 0.25).cuda() if biased else None
    check(l, bias, r, k)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [m.MOE_SCORE_SIGMOID, m.MOE_SCORE_SOFTMAX])
@pytest.mark.parametrize("groups", [(1, 1), (8, 4)])
def test_orders_that_fp32_cannot_tell(score, groups):
    """Scores and biases a fraction of an fp32 step apart: the order is that of the exact sums."""
    E, k = 256, 8
    g = torch.Generator().manual_seed(5)
    T = 200
    # logits in pairs one fp32 step apart, biases that nearly undo the difference of the scores
    base = torch.randn(T, E // 2, generator=g)
    l = torch.stack([base, torch.nextafter(base, torch.tensor(10.0))], 2).view(T, E)
    l = l[:, torch.randperm(E, generator=g)].contiguous()
    bias = (torch.randint(0, 3, (E,), generator=g) * 2.0 ** -26).float()
    r = m.Router(score, groups[0], groups[1], m.MOE_GROUP_TOP2, 1, 1.0)
    check(l.cuda(), bias.cuda(), r, k)
    check(l.cuda(), None, r, k)
    # the whole row within a few steps of one value
    l = (1.0 + torch.randint(0, 40, (T, E), generator=g) * 2.0 ** -23).float()
    check(l.cuda(), bias.cuda(), r, k)


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,r", ROUTERS)
@pytest.mark.parametrize("biased", [False, True])
def test_masked_experts(E, k, r, biased):
    g = torch.Generator().manual_seed(E + 1)
    T = 40
    l = torch.randn(T, E, generator=g) * 2
    l[torch.rand(T, E, generator=g) < 0.3] = -INF
    l[torch.rand(T, E, generator=g) < 0.1] = float("nan")
    l[0] = -INF                      # a row with no expert
    l[1] = float("nan")
    l[2] = -INF
    l[2, E // 2] = 0.5               # one expert left
    l[3] = torch.finfo(torch.float32).min  # the lowest value is a value: all equal
    l[4, ::2] = torch.finfo(torch.float32).min
    bias = (torch.randn(E, generator=g) * 0.1).cuda() if biased else None
    check(l.cuda(), bias, r, k)
    idx, w = call(l.cuda(), bias, r, k)
    assert bool((w[:2] == 0).all()) and bool(torch.isfinite(w).all())
    assert all(len(set(row)) == k and 0 <= min(row) and max(row) < E for row in idx.tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,r", ROUTERS)
@pytest.mark.parametrize("T", [40, 2500])
@pytest.mark.parametrize("low", [-INF, float(torch.finfo(torch.float32).min), -1e4])
def test_biases_that_keep_experts_out(E, k, r, T, low):
    """A bias of -inf, the lowest value or far below the scores: such experts come last, and count as
    what they are where too few others remain."""
    g = torch.Generator().manual_seed(E + T)
    l = (torch.randn(T, E, generator=g) * 1.7).cuda()
    bias = torch.randn(E, generator=g) * 0.05
    bias[torch.rand(E, generator=g) < 0.6] = low
    check(l[:40].contiguous(), bias.cuda(), r, k)
    if T > 40:
        idx, w = call(l, bias.cuda(), r, k)
        i2, w2 = call(l[-40:].contiguous(), bias.cuda(), r, k)
        assert torch.equal(idx[-40:], i2) and bool(((w[-40:] - w2).abs() <= 40 * 2.0 ** -24 * w2).all())


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,r", ROUTERS)
@pytest.mark.parametrize("T", [40, 2500])
@pytest.mark.parametrize("share", [0.05, 0.6, 0.97, 1.0])
def test_nan_biases_keep_experts_out(E, k, r, T, share):
    """Some or all entries of the bias are NaN (a balance update that diverged): as a bias of -inf."""
    g = torch.Generator().manual_seed(E + T)
    l = torch.randn(T, E, generator=g) * 1.7
    l[torch.rand(T, E, generator=g) < 0.1] = -INF
    l = l.cuda()
    bias = torch.randn(E, generator=g) * 0.05
    out = torch.rand(E, generator=g) < share
    low, nan = bias.clone(), bias.clone()
    low[out], nan[out] = -INF, float("nan")
    check(l[:40].contiguous(), low.cuda(), r, k)
    idx, w = call(l, nan.cuda(), r, k)
    i2, w2 = call(l, low.cuda(), r, k)
    assert torch.equal(idx, i2) and torch.equal(w, w2)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [m.MOE_SCORE_SIGMOID, m.MOE_SCORE_SOFTMAX])
@pytest.mark.parametrize("renorm", [0, 1])
def test_large_and_infinite_logits(score, renorm):
    r = m.Router(score, 1, 1, m.MOE_GROUP_MAX, renorm, 1.0)
    l = torch.tensor([[-200.0, -201.0, -202.0, -300.0, -301.0, -400.0, -401.0, -402.0],
                      [30.0, 29.0, 28.0, -5.0, 0.0, 1.0, 2.0, 3.0],
                      [-80.0, -81.0, 2.0, -90.0, -95.0, -99.0, -99.5, -100.0],
                      [INF, 0.0, 1.0, 2.0, -INF, 3.0, 4.0, 5.0]]).cuda()
    idx, w = call(l, None, r, 3)
    ridx, rw, _, _ = reference(l, None, r, 3)
    assert torch.equal(idx.cpu().long(), ridx)
    # arguments up to 402: 402 + 19 roundings; fp32 underflow below 2^-126 is absolute
    assert bool(((w.double().cpu() - rw).abs() <= 430 * 2.0 ** -24 * rw + 2.0 ** -126).all())
    if renorm:
        assert bool(((w.double().sum(1) - 1).abs() < 1e-6).all())


def few_and_many(l, bias, r, k, T):
    """check() on the first 48 rows, and row by row the same in a batch of T."""
    rows = len(l)
    check(l, bias, r, k)
    big = l.repeat((T + rows - 1) // rows, 1)[:T].contiguous()
    idx, w = call(big, bias, r, k)
    i2, w2 = call(l, bias, r, k)
    at = torch.arange(T, device="cuda") % rows
    assert torch.equal(idx, i2[at])
    assert bool(((w - w2[at]).abs() <= 40 * 2.0 ** -24 * w2[at]).all())


@pytest.mark.gpu
def test_an_infinite_logit_keeps_its_group():
    """sigmoid(inf) = 1 and no more: its group has the best expert, and is the one kept."""
    r = m.Router(m.MOE_SCORE_SIGMOID, 8, 1, m.MOE_GROUP_MAX, 1, 1.0)
    l = torch.zeros(5, 64)
    for t, e in enumerate((0, 7, 20, 41, 63)):
        l[t, e] = INF
    for bias in (torch.zeros(64), None):
        idx, _ = call(l.cuda(), None if bias is None else bias.cuda(), r, 3)
        assert idx[:, 0].tolist() == [0, 7, 20, 41, 63]
    # beside a low bias it is one expert among others
    bias = torch.zeros(64)
    bias[20] = -2.0
    check(l.cuda(), bias.cuda(), r, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,r", ROUTERS)
@pytest.mark.parametrize("low", [0.0, -3.0, INF])
def test_infinite_logits_beside_biases(E, k, r, low):
    """Infinite logits among others, beside biases of which some are zero, far down or +inf."""
    g = torch.Generator().manual_seed(E + k)
    l = torch.randn(48, E, generator=g) * 1.7
    l[torch.rand(48, E, generator=g) < 0.03] = INF
    l[torch.rand(48, E, generator=g) < 0.1] = -INF
    bias = torch.randn(E, generator=g) * 0.1
    bias[torch.rand(E, generator=g) < 0.4] = low
    few_and_many(l.cuda(), bias.cuda(), r, k, 2500)


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,r", ROUTERS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_biases_whose_sums_pass_the_largest_float(E, k, r, sign):
    """Two biases of a group add up to more than fp32 holds, and such groups still differ."""
    g = torch.Generator().manual_seed(E + k)
    l = torch.randn(48, E, generator=g) * 1.7
    bias = sign * (1.0 + 2.4 * torch.rand(E, generator=g)) * 1e38
    few_and_many(l.cuda(), bias.cuda(), r, k, 2500)
    bias[torch.rand(E, generator=g) < 0.5] = 0.0
    few_and_many(l.cuda(), bias.cuda(), r, k, 2500)


SATURATED = [(64, 4, 8, 2), (64, 32, 8, 4), (64, 32, 1, 1), (256, 8, 8, 4), (1024, 8, 1, 1), (1024, 32, 1, 1), (96, 6, 32, 7),
             (40, 31, 1, 1), (40, 32, 1, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("score", [m.MOE_SCORE_SIGMOID, m.MOE_SCORE_SOFTMAX])
@pytest.mark.parametrize("E,k,groups,kept", SATURATED)
@pytest.mark.parametrize("T", [24, 2500])
def test_scores_that_saturate(score, E, k, groups, kept, T):
    """Logits whose scores are equal in fp64, in rows that every path decides: without a bias the
    logits order them, with one its fp64 sum does, and equal ones go to the lower expert."""
    g = torch.Generator().manual_seed(E + k)
    values = torch.tensor([40.0, 41.0, 50.0, 60.0, 100.0, 3.0, 2.0, -1.0, -800.0, -900.0])
    l = values[torch.randint(0, len(values), (24, E), generator=g)]
    l[8:16] = torch.where(torch.rand(8, E, generator=g) < 0.9, torch.tensor(40.0), l[8:16])  # more equal ones than candidates
    l[16:] = torch.where(torch.rand(8, E, generator=g) < 0.9, torch.tensor(-INF), l[16:])  # fewer than k unmasked
    l[17] = torch.where(l[17] == -INF, l[17], torch.tensor(INF))
    r = m.Router(score, groups, kept, m.MOE_GROUP_MAX, 1, 1.0)
    gs = E // groups
    want = torch.zeros(24, k, dtype=torch.int64)
    for t, row in enumerate(l.tolist()):
        best = sorted(range(groups), key=lambda i: (-max(row[i * gs:(i + 1) * gs]), i))[:kept]
        want[t] = torch.tensor(sorted((e for i in best for e in range(i * gs, (i + 1) * gs)), key=lambda e: (-row[e], e))[:k])
    big = l.repeat((T + 23) // 24, 1)[:T].contiguous().cuda()
    at = torch.arange(T) % 24
    idx, _ = call(big, None, r, k)
    assert torch.equal(idx.cpu().long(), want[at])
    for bias in (torch.zeros(E), torch.full((E,), 0.25)):
        idx, _ = call(big, bias.cuda(), r, k)
        assert torch.equal(idx.cpu().long(), reference(l, bias, r, k)[0][at])


@pytest.mark.gpu
@pytest.mark.parametrize("score", [m.MOE_SCORE_SIGMOID, m.MOE_SCORE_SOFTMAX])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gradient_against_differences(score, renorm):
    """Central differences of the kernel's own weights, step h = 2^-6: the third derivative of a
    weight is below 1 (h^2 / 6 = 4.1e-5), the two weights are off by 40 * 2^-24 each (/ 2h: 1.5e-4)."""
    E, k, T, h = 16, 4, 12, 2.0 ** -6
    g = torch.Generator().manual_seed(3)
    # logits 0.25 apart in a random order: the selection does not change within h
    l = torch.stack([torch.randperm(E, generator=g).float() * 0.25 - 2 for _ in range(T)]).cuda()
    r = m.Router(score, 1, 1, m.MOE_GROUP_MAX, renorm, 1.0)
    idx, _ = call(l, None, r, k)
    dw = torch.randn(T, k, generator=g).cuda()
    d = torch.empty(T, E, device="cuda")
    m.moe_route_scored_backward(shape_of(E, k), r, T, l, idx, dw, d)
    for e in range(E):
        up, down = l.clone(), l.clone()
        up[:, e] += h
        down[:, e] -= h
        iu, wu = call(up, None, r, k)
        il, wl = call(down, None, r, k)
        assert torch.equal(iu, idx) and torch.equal(il, idx)
        diff = ((wu - wl).double() * dw.double()).sum(1) / (2 * h)
        tol = (4.1e-5 + 1.6e-4) * dw.double().abs().sum(1)
        assert bool(((diff - d[:, e].double()).abs() <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("score", [m.MOE_SCORE_SIGMOID, m.MOE_SCORE_SOFTMAX])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gradients_of_masked_experts_stay_out(score, renorm):
    """Masked experts among the selected, with infinities and NaN for their weights' gradients."""
    E, k, T = 64, 6, 30
    r = m.Router(score, 1, 1, m.MOE_GROUP_MAX, renorm, 1.5)
    g = torch.Generator().manual_seed(4)
    l = torch.randn(T, E, generator=g)
    for t in range(T):
        l[t, torch.randperm(E, generator=g)[:E - t % (k + 1)]] = -INF if t % 2 else float("nan")
    l = l.cuda()
    idx, _ = call(l, None, r, k)
    dw = torch.randn(T, k, generator=g).cuda()
    lk = l.gather(1, idx.long())
    masked = torch.isnan(lk) | (lk == -INF)
    assert bool(masked.any()) and not bool(masked.all())
    want, got = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    m.moe_route_scored_backward(shape_of(E, k), r, T, l, idx, dw.masked_fill(masked, 0.0), want)
    for bad in (float("nan"), INF):
        m.moe_route_scored_backward(shape_of(E, k), r, T, l, idx, dw.masked_fill(masked, bad), got)
        assert torch.equal(got, want) and bool((got[torch.isnan(l) | (l == -INF)] == 0).all())


@pytest.mark.gpu
def test_no_bias_softmax_agrees_with_moe_route():
    E, k, T = 256, 8, 100
    l = (torch.randn(T, E, generator=torch.Generator().manual_seed(1)) * 2).cuda()
    r = m.Router(m.MOE_SCORE_SOFTMAX, 1, 1, m.MOE_GROUP_MAX, 0, 1.0)
    idx, wt = call(l, None, r, k)
    i2, w2 = torch.empty_like(idx), torch.empty_like(wt)
    m.moe_route(shape_of(E, k), T, None, None, None, l, None, i2, w2, None)
    assert torch.equal(idx, i2)
    assert bool(((wt - w2).abs() <= 64 * 2.0 ** -24 * w2).all())


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 33, 700])
def test_from_hidden_states(tokens):
    """Through the router GEMM: the logits are moe_route's, and the selection that of these logits."""
    w = mi.WORKLOADS["tiny"].with_(tokens=tokens, hidden=600, n_experts=72, n_slots=72, top_k=6, n_blocks=8)
    x, wr = mi.hidden_states(w).cuda(), mi.router_weight(w).cuda()
    T, E, k = tokens, 72, 6
    ws = torch.empty(m.moe_route_workspace_size(w, T), dtype=torch.uint8, device="cuda")
    lo, l2 = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    idx, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    r = m.Router(m.MOE_SCORE_SIGMOID, 8, 3, m.MOE_GROUP_TOP2, 1, 2.5)
    bias = torch.linspace(-0.05, 0.05, E).cuda()
    m.moe_route_scored(w, r, T, x, wr, bias, None, lo, idx, wt, ws)
    i2, w2 = torch.empty_like(idx), torch.empty_like(wt)
    m.moe_route(w, T, x, wr, None, None, l2, i2, w2, ws)
    assert m.moe_check_status() == 0
    # the same partial sums; moe_route adds them in groups up to 64 tokens
    assert bool(((lo - l2).abs() <= 2.0 ** -20 * l2.abs().amax()).all())
    ridx, rw, _, _ = reference(lo, bias, r, k)
    assert torch.equal(idx.cpu().long(), ridx)
    assert bool(((wt.double().cpu() - rw).abs() <= 40 * 2.0 ** -24 * rw).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2431, 2432, 5003])
@pytest.mark.parametrize("E,k,r", ROUTERS)
def test_large_batches_match_small_ones(E, k, r, T):
    """Row by row the same whatever the batch (which chooses how many tokens a warp takes)."""
    g = torch.Generator().manual_seed(T + E)
    l = torch.randn(T, E, generator=g) * 1.7
    l[torch.rand(T, E, generator=g) < 0.02] = -INF
    l[::7] = torch.randint(-1, 2, (len(l[::7]), E), generator=g).float()  # ties
    l = l.cuda()
    bias = (torch.randn(E, generator=g) * 0.05).cuda()
    for b in (bias, None):
        idx, w = call(l, b, r, k)
        for a in range(0, T, 600):
            i2, w2 = call(l[a:a + 600].contiguous(), b, r, k)
            assert torch.equal(idx[a:a + 600], i2)
            # a softmax's sum may be added in another order: log2(E) roundings
            assert bool(((w[a:a + 600] - w2).abs() <= 40 * 2.0 ** -24 * w2).all())


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    T, E, k = 2_200_000, 1024, 8
    r = m.Router(m.MOE_SCORE_SOFTMAX, 1, 1, m.MOE_GROUP_MAX, 0, 1.0)
    l = torch.zeros(T, E, device="cuda")
    l[-50:] = torch.randn(50, E, generator=torch.Generator().manual_seed(1)).cuda()
    idx, w = call(l, None, r, k)
    i2, w2 = call(l[-50:].contiguous(), None, r, k)
    assert torch.equal(idx[-50:], i2) and bool(((w[-50:] - w2).abs() <= 40 * 2.0 ** -24 * w2).all())
    assert bool((idx[:-50] == torch.arange(k, device="cuda")).all())
    d = torch.full((T, E), float("nan"), device="cuda")
    dw = torch.ones(T, k, device="cuda")
    m.moe_route_scored_backward(shape_of(E, k), r, T, l, idx, dw, d)
    d2 = torch.empty(50, E, device="cuda")
    m.moe_route_scored_backward(shape_of(E, k), r, 50, l[-50:].contiguous(), i2, dw[:50], d2)
    assert torch.equal(d[-50:], d2) and bool(torch.isfinite(d).all())


@pytest.mark.gpu
def test_out_of_range_ids_in_the_backward_pass_set_the_status():
    r = m.Router(m.MOE_SCORE_SIGMOID, 1, 1, m.MOE_GROUP_MAX, 1, 1.0)
    l = torch.zeros(3, 16, device="cuda")
    idx = torch.tensor([[0, 1], [16, 2], [-1, 3]], dtype=torch.int32, device="cuda")
    d = torch.empty(3, 16, device="cuda")
    m.moe_route_scored_backward(shape_of(16, 2), r, 3, l, idx, torch.ones(3, 2, device="cuda"), d)
    assert m.moe_check_status() == m.MOE_ERR_DEVICE_STATUS
    assert bool(torch.isfinite(d).all()) and m.moe_check_status() == 0


@pytest.mark.gpu
def test_runs_on_another_stream_and_from_a_graph():
    E, k, T = 256, 8, 300
    r = m.Router(m.MOE_SCORE_SIGMOID, 8, 4, m.MOE_GROUP_TOP2, 1, 2.5)
    g = torch.Generator().manual_seed(9)
    l = torch.randn(T, E, generator=g).cuda()
    dw = torch.randn(T, k, generator=g).cuda()
    idx, w = call(l, None, r, k)
    d = torch.empty(T, E, device="cuda")
    m.moe_route_scored_backward(shape_of(E, k), r, T, l, idx, dw, d)
    torch.cuda.synchronize()
    i2, w2, d2 = torch.empty_like(idx), torch.empty_like(w), torch.empty_like(d)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        m.moe_route_scored(shape_of(E, k), r, T, None, None, None, l, None, i2, w2)
        m.moe_route_scored_backward(shape_of(E, k), r, T, l, i2, dw, d2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(d, d2)
    l2 = torch.randn(T, E, generator=g)
    l.copy_(l2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(i2.cpu().long(), reference(l2, None, r, k)[0])


# ------------------------------------------------------------------ refusals (no GPU)
def test_refusals():
    m.build_library()
    L = m.lib()
    b = ctypes.c_void_p(FAKE)
    ok = dict(score=1, n_groups=8, topk_groups=4, group_score=1, renormalize=1, scale=2.5)

    def rc(s=None, T=4, x=None, wr=None, bias=None, lin=b, lout=None, idx=b, w=b, ws=None, n=0, **kw):
        r = m.Router(**{**ok, **kw})
        s = s or shape_of(256, 8)
        return L.moe_route_scored(ctypes.byref(s), ctypes.byref(r), T, x, wr, bias, lin, lout, idx, w, ws, n, None)

    def rcb(T=4, lin=b, idx=b, dw=b, d=b, **kw):
        r = m.Router(**{**ok, **kw})
        s = shape_of(256, 8)
        return L.moe_route_scored_backward(ctypes.byref(s), ctypes.byref(r), T, lin, idx, dw, d, None)

    inv = m.MOE_ERR_INVALID_ARG
    for kw in (dict(score=2), dict(score=-1), dict(group_score=2), dict(renormalize=2), dict(scale=float("nan")),
               dict(scale=INF), dict(n_groups=0), dict(n_groups=3), dict(n_groups=64), dict(topk_groups=0),
               dict(topk_groups=9)):
        assert rc(**kw) == inv and rcb(**kw) == inv, kw
    assert rc(s=shape_of(32, 8), topk_groups=1) == inv and "top_k" in m.last_error()
    assert rc(s=shape_of(8, 9)) == inv and rc(T=-1) == inv
    mis = ctypes.c_void_p(FAKE + 2)
    for kw in (dict(idx=None), dict(w=None), dict(lin=mis), dict(idx=mis), dict(bias=mis), dict(lout=mis)):
        assert rc(**kw) == inv, kw
    for kw in (dict(lin=None), dict(idx=None), dict(dw=None), dict(d=None), dict(d=mis)):
        assert rcb(**kw) == inv, kw
    assert rc(lin=None) == inv and "x" in m.last_error()
    s = shape_of(256, 8, hidden=7168)
    need = m.moe_route_workspace_size(s, 4)
    assert need > 0 and rc(s=s, lin=None, x=b, wr=b, ws=b, n=need - 1) == m.MOE_ERR_WORKSPACE
    assert L.moe_route_scored(ctypes.byref(s), None, 4, None, None, None, b, None, b, b, None, 0, None) == inv
    # nothing to do
    assert rc(T=0, lin=None, idx=None, w=None) == m.MOE_OK and rcb(T=0, lin=None, idx=None, dw=None, d=None) == m.MOE_OK


def test_binding_checks_sizes_and_types():
    r, s = m.Router(), shape_of(16, 2)
    l = torch.zeros(3, 16)
    with pytest.raises(ValueError, match="logits_in"):
        m.moe_route_scored(s, r, 3, None, None, None, l.double(), None, None, None)
    with pytest.raises(ValueError, match="logits_in"):
        m.moe_route_scored(s, r, 4, None, None, None, l, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_route_scored(s, r, 3, None, None, None, l, None, None, None)
    with pytest.raises(ValueError, match="topk_idx"):
        m.moe_route_scored_backward(s, r, 3, None, torch.zeros(3, 2, dtype=torch.int64), None, None)
