"""tenant_forward: scored routing, the experts and the adapters beside the shared
down projection together, against the same layer written out in fp64 (the
intermediates that the layer keeps in bf16 are rounded there too)."""
import pytest
import torch

import moe_expert_layer_06_gb300 as m
import moe_inputs as mi
from moe_expert_layer_06_gb300.tenants import Buffers, shared_down_matrix, tenant_forward
from moe_testlib import assert_close, to_np
from test_scored_route import reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
W = mi.WORKLOADS["tiny"].with_(name="tenants", hidden=256, inter=136, n_experts=16, top_k=4, n_shared=2, inter_shared=72,
                               n_slots=16, n_blocks=4)
ROUTER = m.Router(m.MOE_SCORE_SIGMOID, 4, 2, m.MOE_GROUP_TOP2, 1, 2.5)


def inputs(T, n=5, r=16, seed=0):
    w = W.with_(tokens=T)
    g = torch.Generator().manual_seed(seed + T)
    t = dict(zip(("wg", "wu", "wd"), mi.stacked_expert_weights(w)))
    t.update(zip(("sg", "su", "sd"), mi.stacked_shared_weights(w)))
    t.update(x=mi.hidden_states(w), wr=mi.router_weight(w), bias=torch.randn(w.n_experts, generator=g) * 0.1)
    K = w.n_shared * w.inter_shared
    t.update(a=(torch.randn(n, r, K, generator=g) * K ** -0.5).bfloat16(),
             b=(torch.randn(n, w.hidden, r, generator=g) * r ** -0.5).bfloat16(),
             s=torch.rand(n, generator=g) + 0.5, of=torch.randint(-1, n, (T,), generator=g).int())
    return w, m.Adapter(K, w.hidden, n, r), t


def by_hand(w, t, idx, wt):
    """The layer in fp64 with the routing given."""
    T = t["x"].shape[0]
    d = {k: v.double() for k, v in t.items() if k != "of"}
    bf = lambda v: v.to(torch.bfloat16).double()  # noqa: E731

    def ffn_h(x, g, u):
        a, b = x @ g.t(), x @ u.t()
        return bf(a / (1.0 + torch.exp(-a)) * b)

    out = torch.zeros(T, w.hidden).double()
    for tok in range(T):
        for j in range(w.top_k):
            e = int(idx[tok, j])
            y = bf(ffn_h(d["x"][tok:tok + 1], d["wg"][e], d["wu"][e]) @ d["wd"][e].t())
            out[tok] += wt[tok, j] * y[0]
    hs = torch.cat([ffn_h(d["x"], d["sg"][j], d["su"][j]) for j in range(w.n_shared)], 1)
    out += hs @ shared_down_matrix(t["sd"]).double().t()
    for tok in range(T):
        i = int(t["of"][tok])
        if i >= 0:
            out[tok] += d["b"][i] @ bf(d["s"][i] * (d["a"][i] @ hs[tok]))
    return out


@pytest.mark.parametrize("T", [1, 16, 50, 300])
def test_against_the_layer_in_fp64(T):
    w, ad, t = inputs(T)
    d = {k: v.to(DEV) for k, v in t.items()}
    buf = Buffers(w, ad, T)
    out = torch.empty(T, w.hidden, dtype=torch.bfloat16, device=DEV)

    def forward():
        tenant_forward(w, ROUTER, ad, T, d["x"], d["wr"], d["bias"], d["wg"], d["wu"], d["wd"], d["sg"], d["su"],
                       shared_down_matrix(d["sd"]), d["a"], d["b"], d["s"], d["of"], out, buf)

    forward()
    assert m.moe_check_status() == 0
    # the routing of the kernel's own logits (their error could swap near neighbours)
    logits = torch.empty(T, w.n_experts, device=DEV)
    idx, wt = torch.empty_like(buf.topk_idx), torch.empty_like(buf.topk_w)
    m.moe_route_scored(w, ROUTER, T, d["x"], d["wr"], d["bias"], None, logits, idx, wt,
                       torch.empty(m.moe_route_workspace_size(w, T), dtype=torch.uint8, device=DEV))
    ridx, rw, _, _ = reference(logits, d["bias"], ROUTER, w.top_k)
    assert torch.equal(buf.topk_idx.cpu().long(), ridx) and torch.equal(buf.topk_idx, idx)
    assert_close(to_np(out), by_hand(w, t, ridx, rw).numpy(), what="tenant layer")


def test_replays_from_a_graph_and_changes_tenants():
    T = 40
    w, ad, t = inputs(T)
    d = {k: v.to(DEV) for k, v in t.items()}
    down = shared_down_matrix(d["sd"])
    buf = Buffers(w, ad, T)
    out = torch.empty(T, w.hidden, dtype=torch.bfloat16, device=DEV)

    def forward(o):
        tenant_forward(w, ROUTER, ad, T, d["x"], d["wr"], d["bias"], d["wg"], d["wu"], d["wd"], d["sg"], d["su"], down,
                       d["a"], d["b"], d["s"], d["of"], o, buf)

    forward(out)
    torch.cuda.synchronize()
    again = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(again)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    d["of"].copy_(torch.randint(-1, 5, (T,), generator=torch.Generator().manual_seed(77)).int())
    graph.replay()
    forward(out)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    assert m.moe_check_status() == 0


@pytest.mark.parametrize("T", [70, 300])
def test_layers_one_after_another(T):
    """The rank product may start while the layer's GEMM before it runs, and that GEMM while the call
    before ends: pass after pass the same."""
    w, ad, t = inputs(T)
    d = {k: v.to(DEV) for k, v in t.items()}
    down, buf = shared_down_matrix(d["sd"]), Buffers(w, ad, T)
    outs = [torch.empty(T, w.hidden, dtype=torch.bfloat16, device=DEV) for _ in range(20)]
    for out in outs:
        tenant_forward(w, ROUTER, ad, T, d["x"], d["wr"], d["bias"], d["wg"], d["wu"], d["wd"], d["sg"], d["su"], down,
                       d["a"], d["b"], d["s"], d["of"], out, buf)
    assert m.moe_check_status() == 0
    assert all(torch.equal(o, outs[0]) for o in outs) and bool(torch.isfinite(outs[0].float()).all())


def test_sizes_that_do_not_belong_together_are_refused():
    w, ad, t = inputs(4)
    with pytest.raises(ValueError, match="features"):
        tenant_forward(w, ROUTER, m.Adapter(8, 8, 1, 8), 4, *[None] * 14, Buffers(w, ad, 4))
    with pytest.raises(ValueError, match="tokens"):
        tenant_forward(w, ROUTER, ad, 5, *[None] * 14, Buffers(w, ad, 4))
