"""training.layer_forward and layer_backward: the operators that train the experts as one layer, against
the same layer written out in fp64 (what the layer keeps in bf16 or in 8 bits is rounded there too)."""
import pytest
import torch

import moe_expert_layer_06_gb300 as m
import moe_inputs as mi
from moe_expert_layer_06_gb300.tenants import shared_down_matrix
from moe_expert_layer_06_gb300.training import Buffers, layer_backward, layer_forward
from moe_testlib import assert_close, to_np
from test_expert_training import kept

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16
W = mi.WORKLOADS["tiny"].with_(name="training", hidden=256, inter=136, n_experts=16, top_k=4, n_shared=2, inter_shared=72,
                               n_slots=16, n_blocks=4)
ROUTER = m.Router(m.MOE_SCORE_SIGMOID, 4, 2, m.MOE_GROUP_TOP2, 1, 2.5)
NAMES = ("wr", "wg", "wu", "wd", "sg", "su", "sd")


def inputs(w):
    t = dict(zip(("wg", "wu", "wd"), mi.stacked_expert_weights(w)))
    if w.n_shared:
        sg, su, sd = mi.stacked_shared_weights(w)
        t.update(sg=sg, su=su, sd=shared_down_matrix(sd))
    g = torch.Generator().manual_seed(w.tokens)
    t.update(x=mi.hidden_states(w), wr=mi.router_weight(w), bias=torch.randn(w.n_experts, generator=g) * 0.1,
             dout=torch.randn(w.tokens, w.hidden, generator=g).to(BF))
    return t


class Layer:
    def __init__(self, w, dtype=BF):
        self.w, self.t = w, inputs(w)
        self.d = {k: v.to(DEV) for k, v in self.t.items()}
        self.b = Buffers(w, w.tokens)
        self.out, self.dx = (torch.full((w.tokens, w.hidden), float("nan"), dtype=BF, device=DEV) for _ in range(2))
        self.grads = {k: torch.full(self.t[k].shape, float("nan"), dtype=dtype, device=DEV) for k in NAMES if k in self.t}

    def forward(self):
        d = self.d
        layer_forward(self.w, ROUTER, self.w.tokens, d["x"], d["wr"], d["bias"], d["wg"], d["wu"], d["wd"], d.get("sg"), d.get("su"),
                      d.get("sd"), self.out, self.b)

    def backward(self, add=False):
        d, g = self.d, self.grads
        layer_backward(self.w, ROUTER, self.w.tokens, d["dout"], d["x"], d["wr"], d["wg"], d["wu"], d["wd"], d.get("sg"), d.get("su"),
                       d.get("sd"), self.dx, g["wr"], g["wg"], g["wu"], g["wd"], g.get("sg"), g.get("su"), g.get("sd"), self.b, add)


def by_hand(w, t, idx):
    """(out, dx, gradients) in fp64 for the selection idx, rounded where the layer rounds."""
    bf = lambda v: v.to(BF).double()  # noqa: E731
    keep = lambda v: kept(v.to(BF))[2].double()  # noqa: E731
    d = {k: v.double() for k, v in t.items()}
    x, T, k = d["x"], w.tokens, w.top_k
    # weights of the selection (renormalised sigmoids), with their gradient
    lg = (x @ d["wr"].t()).requires_grad_(True)
    s = torch.sigmoid(lg).gather(1, idx)
    topw = 2.5 * s / s.sum(1, keepdim=True)

    def act(g, u):
        return g * torch.sigmoid(g) * u

    def ffn(xr, wg, wu, wd, dy):
        """y, and a function of dy: (dx, dwg, dwu, dwd, with x as `xk` for the gradients)"""
        g, u = bf(xr @ wg.t()), bf(xr @ wu.t())
        y = bf(act(g, u)) @ wd.t()
        # (the kept values of a row's gate and up in blocks of their own)
        kg, ku = keep(g), keep(u)

        def back(dy, xk):
            dh = bf(dy @ wd)
            sg = torch.sigmoid(kg)
            dg, du = bf(dh * ku * sg * (1.0 + kg * (1.0 - sg))), bf(dh * kg * sg)
            return dg @ wg + du @ wu, dg.t() @ xk, du.t() @ xk, dy.t() @ bf(act(kg, ku))
        return y, back

    out = torch.zeros_like(x)
    dx, g = torch.zeros_like(x), {n: torch.zeros_like(d[n]) for n in NAMES if n in d}
    dtop = torch.zeros(T, k).double()
    dout = d["dout"]
    xk = keep(x)
    for e in range(w.n_experts):
        tok, j = torch.nonzero(idx == e, as_tuple=True)
        if not tok.numel():
            continue
        y, back = ffn(x[tok], d["wg"][e], d["wu"][e], d["wd"][e], None)
        y = bf(y)
        wt = topw.detach().float().double()[tok, j][:, None]
        out[tok] += wt * y
        dtop[tok, j] = (dout[tok] * y).sum(1)
        dxe, g["wg"][e], g["wu"][e], g["wd"][e] = back(bf(wt * dout[tok]), xk[tok])
        dx[tok] += bf(dxe)
    topw.backward(dtop)
    dl = bf(lg.grad)
    dx += dl @ d["wr"]
    g["wr"] = dl.t() @ x
    if w.n_shared:
        Is = w.n_shared * w.inter_shared
        y, back = ffn(x, d["sg"].view(Is, -1), d["su"].view(Is, -1), d["sd"], None)
        out += y
        dxs, dsg, dsu, g["sd"] = back(dout, x)
        dx += dxs
        g["sg"], g["su"] = dsg.view_as(d["sg"]), dsu.view_as(d["su"])
    return out, dx, g


@pytest.mark.parametrize("T,n_shared", [(1, 2), (50, 2), (300, 2), (129, 0)])
def test_against_the_layer_in_fp64(T, n_shared):
    w = W.with_(tokens=T, n_shared=n_shared, inter_shared=72 if n_shared else 0)
    a = Layer(w)
    a.forward()
    a.backward()
    assert m.moe_check_status() == 0
    out, dx, g = by_hand(w, a.t, a.b.topk_idx.cpu().long())
    assert_close(to_np(a.out), out.numpy(), what="out")
    assert_close(to_np(a.dx), dx.numpy(), what="dx")
    for n in g:
        assert_close(to_np(a.grads[n]).reshape(-1, a.grads[n].shape[-1]), g[n].reshape(-1, g[n].shape[-1]).numpy(), what="d " + n)


def test_added_gradients_replay_and_repeat():
    """Gradients of two batches added in fp32; the step captured in a graph; the same bits again."""
    w = W.with_(tokens=70)
    a = Layer(w, torch.float32)
    a.forward()
    a.backward()
    once = {n: g.clone() for n, g in a.grads.items()}
    out, dx = a.out.clone(), a.dx.clone()
    a.backward(add=True)
    for n, g in a.grads.items():
        assert bool(((g - 2 * once[n]).abs() <= 2.0 ** -22 * once[n].abs() + 1e-30).all()), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.forward()
        a.backward()
    a.out.zero_(), a.dx.zero_()
    for g in a.grads.values():
        g.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert m.moe_check_status() == 0
    assert torch.equal(a.out, out) and torch.equal(a.dx, dx)
    for n, g in a.grads.items():
        assert torch.equal(g, once[n]), n


def test_refusals():
    w = W.with_(tokens=8)
    a = Layer(w)
    a.b = Buffers(w, 9)
    with pytest.raises(ValueError):
        a.forward()
    a = Layer(w.with_(n_experts=12, n_slots=12))
    with pytest.raises(ValueError):
        a.forward()
