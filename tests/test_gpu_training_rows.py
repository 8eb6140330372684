"""training.Buffers(keep_rows=False): the dispatched rows gathered again from x in the backward pass."""
import pytest
import torch

import moe_expert_layer_06_gb300 as m
import test_gpu_training as base
from moe_expert_layer_06_gb300.training import Buffers
from moe_testlib import assert_close, to_np

pytestmark = pytest.mark.gpu


def layer(w, dtype=base.BF):
    a = base.Layer(w, dtype)
    a.b = Buffers(w, w.tokens, keep_rows=False)
    return a


@pytest.mark.parametrize("T,n_shared", [(1, 2), (50, 2), (300, 2), (129, 0)])
def test_against_the_layer_in_fp64(T, n_shared, monkeypatch):
    w = base.W.with_(tokens=T, n_shared=n_shared, inter_shared=72 if n_shared else 0)
    a, kept = layer(w), base.Layer(w)
    for one in (a, kept):
        one.forward()
        one.backward()
    assert m.moe_check_status() == 0
    # everything but the gradients of gate and up is as with kept rows, bit for bit
    assert torch.equal(a.out, kept.out) and torch.equal(a.dx, kept.dx)
    for n in a.grads:
        assert n in ("wg", "wu") or torch.equal(a.grads[n], kept.grads[n]), n
    # and those are of x itself: the reference rounds gate and up, not x
    rounded = base.kept
    monkeypatch.setattr(base, "kept", lambda v: (None, None, v) if v.shape == a.t["x"].shape and torch.equal(v, a.t["x"]) else rounded(v))
    _, _, g = base.by_hand(w, a.t, a.b.topk_idx.cpu().long())
    for n in g:
        assert_close(to_np(a.grads[n]).reshape(-1, a.grads[n].shape[-1]), g[n].reshape(-1, g[n].shape[-1]).numpy(), what="d " + n)


def test_replayed_added_and_on_another_stream():
    w = base.W.with_(tokens=70)
    a = layer(w, torch.float32)
    a.forward()
    a.backward()
    once = {n: g.clone() for n, g in a.grads.items()}
    a.backward(add=True)
    for n, g in a.grads.items():
        assert bool(((g - 2 * once[n]).abs() <= 2.0 ** -22 * once[n].abs() + 1e-30).all()), n
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        a.forward()
        a.backward()
    for g in a.grads.values():
        g.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, once[n]) for n, g in a.grads.items()) and m.moe_check_status() == 0


@pytest.mark.parametrize("keep_rows", [True, False])
def test_no_tokens(keep_rows):
    w = base.W.with_(tokens=1)
    a = base.Layer(w)
    a.w = w.with_(tokens=0)
    a.b = Buffers(a.w, 0, keep_rows=keep_rows)
    for n in ("x", "dout"):
        a.d[n] = a.d[n][:0]
    a.out, a.dx = a.out[:0], a.dx[:0]
    a.forward()
    a.backward()
    assert m.moe_check_status() == 0
    assert all(bool((g == 0).all()) for g in a.grads.values())
