"""training.layer_forward and layer_backward on streams of the caller's."""
import pytest
import torch

import moe_expert_layer_06_gb300 as m
from moe_expert_layer_06_gb300.training import Buffers, layer_backward, layer_forward
from test_gpu_training import BF, DEV, NAMES, ROUTER, W, inputs

pytestmark = pytest.mark.gpu


def outputs(w, t):
    new = lambda shape: torch.full(shape, float("nan"), dtype=BF, device=DEV)  # noqa: E731
    return [new((w.tokens, w.hidden)), new((w.tokens, w.hidden)), {k: new(t[k].shape) for k in NAMES}]


def both(w, d, b, out, dx, g, stream=None):
    T, weights = w.tokens, [d[k] for k in NAMES]
    layer_forward(w, ROUTER, T, d["x"], d["wr"], d["bias"], *weights[1:], out, b, stream=stream)
    layer_backward(w, ROUTER, T, d["dout"], d["x"], *weights, dx, *(g[k] for k in NAMES), b, stream=stream)


def same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])


def test_a_stream_of_its_own():
    """Buffers made behind work of the current stream, passes on another one (a Stream or its handle) that waits for nothing."""
    w = W.with_(tokens=90)
    t = inputs(w)
    d = {k: v.to(DEV) for k, v in t.items()}
    want = outputs(w, t)
    both(w, d, Buffers(w, 90), *want)
    torch.cuda.synchronize()
    for raw in (False, True):
        side, got = torch.cuda.Stream(), outputs(w, t)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # some 10 ms of the current stream
        b = Buffers(w, 90)
        torch.cuda._sleep(20_000_000)
        both(w, d, b, *got, stream=side.cuda_stream if raw else side)
        side.synchronize()
        assert same(got, want)
        torch.cuda.synchronize()
    assert m.moe_check_status() == 0


def test_two_layers_at_once():
    """Two streams, buffers of their own, several passes beside each other: the bits of passes alone."""
    w = W.with_(tokens=200)
    t = inputs(w)
    d = {k: v.to(DEV) for k, v in t.items()}
    want = outputs(w, t)
    both(w, d, Buffers(w, 200), *want)
    sides, got = [torch.cuda.Stream() for _ in range(2)], [outputs(w, t) for _ in range(2)]
    bufs = [Buffers(w, 200) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for side, b, o in zip(sides, bufs, got):
            both(w, d, b, *o, stream=side)
    torch.cuda.synchronize()
    assert same(got[0], want) and same(got[1], want)
    assert m.moe_check_status() == 0
