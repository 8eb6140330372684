"""Low-rank adapters beside a shared projection (moe_adapter_project and its
backward pass) against their definition in 64 bits.

Tolerances, element by element.  An output rounds once to bf16 (half a step:
2^-8 of its value); v and dv round once (2^-8 of theirs, through the other
adapter matrix); every fp32 sum of n products is off by at most n steps of
2^-23 of the sum of their magnitudes (2^-24 for a rounded sum; twice that
where a tensor core truncates)."""
import ctypes

import pytest
import torch

import moe_expert_layer_06_gb300 as m

FAKE = 0x10000  # aligned address that is never dereferenced on the host
HALF = 2.0 ** -8
STEP = 2.0 ** -23


class Case:
    def __init__(self, T, K, N, r, n, ids="each", scaled=True, seed=0):
        g = torch.Generator().manual_seed(seed + 31 * T + K + N + r)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)

        self.T, self.K, self.N, self.r, self.n = T, K, N, r, n
        self.p = m.Adapter(K, N, n, r)
        self.x, self.dy = normal(T, K), normal(T, N)
        self.w = normal(N, K, std=K ** -0.5)
        self.a, self.b = normal(n, r, K, std=K ** -0.5), normal(n, N, r, std=r ** -0.5)
        self.s = torch.rand(n, generator=g) + 0.5 if scaled else None
        if ids == "each":
            self.of = torch.randint(-1, n, (T,), generator=g)
        elif ids == "runs":
            self.of = (torch.arange(T) // 50) % (n + 1) - 1
        elif ids == "none":
            self.of = torch.full((T,), -1)
        else:
            self.of = torch.full((T,), n - 1)
        self.of = self.of.to(torch.int32)

    def dev(self, t):
        return None if t is None else t.cuda()

    def forward(self, fp32=False, want_v=True, ws=None):
        out = torch.full((self.T, self.N), float("nan"), dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        v = torch.full((self.T, self.r), float("nan"), dtype=torch.bfloat16, device="cuda") if want_v else None
        ws = scratch(self.p, self.T) if ws is None else ws
        m.moe_adapter_project(self.p, self.T, self.dev(self.x), self.dev(self.w), self.dev(self.a), self.dev(self.b),
                              self.dev(self.s), self.dev(self.of), out, v, ws)
        return out, v

    def backward(self, v, dx=True, grads=True):
        new = lambda *shape: torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        dx = new(self.T, self.K) if dx else None
        da, db = (new(self.n, self.r, self.K), new(self.n, self.N, self.r)) if grads else (None, None)
        m.moe_adapter_project_backward(self.p, self.T, self.dev(self.dy), self.dev(self.x), self.dev(self.w),
                                       self.dev(self.a), self.dev(self.b), self.dev(self.s), self.dev(self.of), v, dx, da,
                                       db, scratch(self.p, self.T))
        return dx, da, db

    def reference(self):
        """Values and tolerances of (y, v, dx, da, db), fp64."""
        x, dy, w, a, b = (t.double() for t in (self.x, self.dy, self.w, self.a, self.b))
        T, K, N, r = self.T, self.K, self.N, self.r
        y, ey = x @ w.t(), K * STEP * (x.abs() @ w.abs().t())
        dx, edx = dy @ w, N * STEP * (dy.abs() @ w.abs())
        v, ev = torch.zeros(T, r).double(), torch.zeros(T, r).double()
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        eda, edb = torch.zeros_like(a), torch.zeros_like(b)
        for i in range(self.n):
            rows = torch.nonzero(self.of == i).flatten()
            if not rows.numel():
                continue
            s = float(self.s[i]) if self.s is not None else 1.0
            xi, di, ai, bi = x[rows], dy[rows], a[i], b[i]
            vi, dvi = s * (xi @ ai.t()), s * (di @ bi)
            # v before and after its rounding
            evi = HALF * vi.abs() + 2 * K * STEP * s * (xi.abs() @ ai.abs().t())
            edvi = HALF * dvi.abs() + 2 * N * STEP * s * (di.abs() @ bi.abs())
            y[rows] += vi @ bi.t()
            ey[rows] += (evi + r * STEP * vi.abs()) @ bi.abs().t()
            dx[rows] += dvi @ ai
            edx[rows] += (edvi + r * STEP * dvi.abs()) @ ai.abs()
            v[rows], ev[rows] = vi, evi
            n = rows.numel()
            da[i], eda[i] = dvi.t() @ xi, (edvi + n * STEP * dvi.abs()).t() @ xi.abs()
            db[i], edb[i] = di.t() @ vi, di.abs().t() @ (evi + n * STEP * vi.abs())
        return {"y": (y, ey), "v": (v, ev), "dx": (dx, edx), "da": (da, eda), "db": (db, edb)}


def scratch(p, T):
    return torch.empty(max(256, m.moe_adapter_workspace_size(p, T)), dtype=torch.uint8, device="cuda")


def close(got, want, tol, bf16=True, name=""):
    got = got.double().cpu()
    tol = tol + (HALF * want.abs() + HALF * tol if bf16 else 2.0 ** -23 * want.abs()) + 1e-30
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (name, int(bad.sum()), float(((got - want).abs() / tol).max()))


# (K, N, rank, adapters): every dimension ragged somewhere, ranks of one to four 64-wide chunks
SIZES = [(64, 128, 8, 1), (72, 136, 16, 3), (600, 328, 24, 5), (1000, 616, 64, 40), (256, 512, 72, 2), (520, 264, 256, 3),
         (8, 8, 8, 2), (2048, 1024, 32, 7)]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 17, 33, 64, 65, 129, 257, 700])
@pytest.mark.parametrize("K,N,r,n", SIZES)
def test_forward_matches_the_definition(T, K, N, r, n):
    for ids in ("each", "runs"):
        c = Case(T, K, N, r, n, ids)
        y, v = c.forward()
        assert m.moe_check_status() == 0
        ref = c.reference()
        close(y, *ref["y"], name="y " + ids)
        # ev has the rounding of v already
        assert bool(((v.double().cpu() - ref["v"][0]).abs() <= 1.01 * ref["v"][1] + 1e-30).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 33, 64, 129, 257, 700])
@pytest.mark.parametrize("K,N,r,n", SIZES)
def test_backward_matches_the_definition(T, K, N, r, n):
    for ids in ("each", "runs", "one"):
        c = Case(T, K, N, r, n, ids)
        _, v = c.forward()
        dx, da, db = c.backward(v)
        assert m.moe_check_status() == 0
        ref = c.reference()
        close(dx, *ref["dx"], name="dx " + ids)
        close(da, *ref["da"], name="da " + ids)
        close(db, *ref["db"], name="db " + ids)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r,n", [(1500, 136, 8200, 24, 3), (1100, 8200, 264, 40, 2), (2100, 264, 520, 16, 700)])
def test_more_tiles_than_processors_and_many_adapters_per_tile(T, K, N, r, n):
    """Forward and backward with several tiles per CTA, and with nearly every token's adapter its own."""
    for ids in ("runs", "each"):
        c = Case(T, K, N, r, n, ids)
        y, v = c.forward()
        dx, da, db = c.backward(v)
        assert m.moe_check_status() == 0
        ref = c.reference()
        for name, got in (("y", y), ("dx", dx), ("da", da), ("db", db)):
            close(got, *ref[name], name=name + " " + ids)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r,n", [(100, 264, 24008, 24, 3), (200, 24008, 136, 8, 5), (2040, 264, 1000, 16, 9),
                                       (1100, 2104, 1000, 32, 2), (300, 72, 5000, 64, 4)])
def test_tiles_that_no_cluster_shares(T, K, N, r, n):
    """Outputs through shared memory, at every tile height, feature and token edge."""
    c = Case(T, K, N, r, n, "each")
    ref = c.reference()
    y, v = c.forward()
    close(y, *ref["y"], name="y")
    dx, da, db = c.backward(v)
    for got, name in ((dx, "dx"), (da, "da"), (db, "db")):
        close(got, *ref[name], name=name)


@pytest.mark.gpu
@pytest.mark.parametrize("T,long,short,n", [(956, 7720, 216, 5), (2048, 9000, 136, 6), (300, 2048, 72, 40), (9000, 520, 200, 3)])
def test_calls_one_after_another_over_a_short_contraction(T, long, short, n):
    """A short rank product may start while the projection of the call before it runs."""
    new = lambda *shape: torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for c in (Case(T, short, long, 24, n), Case(T, long, short, 24, n)):
        x, w, a, b, s, of, dy = (t.cuda() for t in (c.x, c.w, c.a, c.b, c.s, c.of, c.dy))
        ws, outs = scratch(c.p, T), []
        for _ in range(12):
            if c.N == long:
                out = [new(T, c.N), new(T, 24)]
                m.moe_adapter_project(c.p, T, x, w, a, b, s, of, *out, ws)
            else:
                out = [new(T, c.K), new(n, 24, c.K), new(n, c.N, 24)]
                m.moe_adapter_project_backward(c.p, T, dy, x, w, a, b, s, of, x[:, :24].contiguous(), *out, ws)
            outs.append(out)
        assert m.moe_check_status() == m.MOE_OK
        for out in outs:
            assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(out, outs[0]))
        assert all(bool(torch.isfinite(t).all()) for t in outs[0])


@pytest.mark.gpu
@pytest.mark.parametrize("C", [64, 192, 256, 448])
@pytest.mark.parametrize("T,r,n", [(1, 64, 16), (16, 64, 16), (64, 64, 64), (200, 72, 64), (300, 256, 16)])
@pytest.mark.parametrize("ids", ["none", "one", "two"])
def test_short_contractions_with_few_of_many_adapters(T, C, r, n, ids):
    """Fewer chunks of contraction than the clusters that the configured adapters call for have CTAs, and
    a batch that uses none, one or two of those: some CTAs have nothing to multiply."""
    loud = Case(256, 512, 4096, 8, 1, "none")  # leaves large sums in the tensor memory
    loud.x *= 1000
    for K, N in ((C, 1024), (1024, C)):
        c = Case(T, K, N, r, n, "none" if ids == "none" else "one")
        if ids == "two":
            c.of[::2] = 0
        ref = c.reference()
        loud.forward()
        y, v = c.forward()
        y32, _ = c.forward(fp32=True)
        loud.forward()
        dx, da, db = c.backward(v)
        assert m.moe_check_status() == 0
        close(y32, *ref["y"], bf16=False, name="y fp32")
        for name, got in (("y", y), ("dx", dx), ("da", da), ("db", db)):
            close(got, *ref[name], name=name)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r,n", [(7, 2056, 136, 8, 2), (150, 1160, 2184, 72, 1), (520, 2312, 264, 24, 1)])
def test_shared_sums_past_the_last_feature_and_rank(T, K, N, r, n):
    """Clusters whose CTAs read one another's sums, where tiles reach past the features and the rank:
    call after call the same."""
    c = Case(T, K, N, r, n, "one")
    ref = c.reference()
    x, w, a, b, s, of, dy = (t.cuda() for t in (c.x, c.w, c.a, c.b, c.s, c.of, c.dy))
    ws, outs = scratch(c.p, T), []
    new = lambda *shape: torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for _ in range(10):
        y, v, dx, da, db = new(T, N), new(T, r), new(T, K), new(n, r, K), new(n, N, r)
        m.moe_adapter_project(c.p, T, x, w, a, b, s, of, y, v, ws)
        m.moe_adapter_project_backward(c.p, T, dy, x, w, a, b, s, of, v, dx, da, db, ws)
        outs.append((y, v, dx, da, db))
    assert m.moe_check_status() == 0
    for out in outs:
        assert all(torch.equal(p, q) for p, q in zip(out, outs[0]))
    for name, got in zip(("y", "v", "dx", "da", "db"), outs[0]):
        close(got, *ref[name], name=name)


@pytest.mark.gpu
def test_very_long_batches():
    """More 64-token chunks than the gradient kernel lists at a time (262144 tokens)."""
    c = Case(270001, 16, 24, 8, 3, "runs")
    y, v = c.forward()
    dx, da, db = c.backward(v)
    assert m.moe_check_status() == 0
    ref = c.reference()
    for name, got in (("y", y), ("dx", dx), ("da", da), ("db", db)):
        close(got, *ref[name], name=name)


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """An output of more than 2^31 elements: its last rows are those of the last tokens alone."""
    T, K, N, r, n, tail = 270000, 8, 8200, 8, 2, 100
    c = Case(tail, K, N, r, n, "each")
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    of = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    x[-tail:], of[-tail:] = c.x.cuda(), c.of.cuda()
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    m.moe_adapter_project(c.p, T, x, c.w.cuda(), c.a.cuda(), c.b.cuda(), c.s.cuda(), of, out, None, scratch(c.p, T))
    assert m.moe_check_status() == 0
    close(out[-tail:], *c.reference()["y"])
    assert not bool(out[:-tail].any())


@pytest.mark.gpu
def test_a_contraction_whose_copies_pass_32_bits():
    """A share of the contraction of more than 2^31 bytes of copies; all but 64 of its features are zero."""
    T, K, N, r = 65, 59_700_000, 8, 8
    c = Case(T, 64, N, r, 1, "one")
    at = torch.cat([torch.arange(32), torch.arange(K - 32, K)])
    big = []
    for t in (c.x, c.w, c.a):
        z = torch.zeros(*t.shape[:-1], K, dtype=torch.bfloat16, device="cuda")
        z[..., at.cuda()] = t.cuda()
        big.append(z)
    p = m.Adapter(K, N, 1, r)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    m.moe_adapter_project(p, T, big[0], big[1], big[2], c.b.cuda(), c.s.cuda(), c.of.cuda(), y, None, scratch(p, T))
    assert m.moe_check_status() == 0
    close(y, *c.reference()["y"])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 300])
def test_no_adapters_no_scaling_and_fp32_output(T):
    c = Case(T, 264, 392, 16, 4, "none", scaled=False)
    y, v = c.forward()
    close(y, *c.reference()["y"])
    assert bool((v == 0).all())
    dx, da, db = c.backward(v)
    close(dx, *c.reference()["dx"])
    assert bool((da == 0).all()) and bool((db == 0).all())
    c = Case(T, 264, 392, 16, 4, "each", scaled=False)
    y, _ = c.forward(fp32=True, want_v=False)
    close(y, *c.reference()["y"], bf16=False)
    y16, _ = c.forward()
    assert torch.equal(y.to(torch.bfloat16), y16)


@pytest.mark.gpu
def test_optional_outputs_and_empty_batches():
    c = Case(70, 264, 392, 16, 4)
    _, v = c.forward()
    dx, da, db = c.backward(v)
    dx1, _, _ = c.backward(None, grads=False)
    _, da1, db1 = c.backward(v, dx=False)
    assert torch.equal(dx, dx1) and torch.equal(da, da1) and torch.equal(db, db1)
    e = Case(0, 264, 392, 16, 4)
    y, v = e.forward()
    _, da, db = e.backward(v)
    assert y.shape == (0, 392) and bool((da == 0).all()) and bool((db == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 64, 300])
def test_infinities_and_nan_stay_with_their_own_request(T):
    """One tenant's adapter or tokens hold infinities and NaN: every other token's results, and every
    other adapter's gradients, are those of a batch without them."""
    c = Case(T, 264, 392, 72, 4, "each", seed=3)
    c.of[:3] = torch.tensor([0, 1, -1], dtype=torch.int32)
    y0, v0 = c.forward()
    g0 = c.backward(v0)
    d = Case(T, 264, 392, 72, 4, "each", seed=3)
    d.of = c.of
    d.b[1, 5, 70] = float("inf")
    d.b[1, 200, 3] = float("nan")
    d.b[1, 391, 0] = float("-inf")
    d.a[1, 7, 100] = float("nan")
    d.a[1, 70, 263] = float("inf")
    d.x[2], d.dy[2] = float("nan"), float("inf")   # a token without adapter (padding)
    y1, v1 = d.forward()
    g1 = d.backward(v1)
    assert m.moe_check_status() == 0
    others = (c.of != 1)
    others[2] = False
    o = others.cuda()
    assert torch.equal(y0[o], y1[o]) and torch.equal(v0[o], v1[o]) and torch.equal(g0[0][o], g1[0][o])
    for i in (0, 2, 3):
        assert torch.equal(g0[1][i], g1[1][i]) and torch.equal(g0[2][i], g1[2][i])
    # and where they belong they show
    mine = (c.of == 1).cuda()
    assert not bool(torch.isfinite(v1[mine].float()).any(1).all()) or bool(torch.isnan(y1[mine].float()).any(1).all())
    assert bool(torch.isnan(y1[2].float()).all())
    # an infinity alone, with finite v, gives infinities of its sign in its own column
    e = Case(T, 264, 392, 72, 4, "each", seed=3)
    e.of = c.of
    e.b[1, 5, 70] = float("inf")
    y2, v2 = e.forward()
    rows = torch.nonzero(mine).flatten()
    want = torch.where(v2[rows, 70] > 0, float("inf"), -float("inf"))
    assert torch.equal(y2[rows, 5].float(), want.float())
    keep = torch.ones(392, dtype=torch.bool)
    keep[5] = False
    assert torch.equal(y2[:, keep.cuda()], y0[:, keep.cuda()])


@pytest.mark.gpu
@pytest.mark.parametrize("T,r", [(5, 16), (64, 72), (300, 72), (2100, 24)])
def test_infinite_products_of_infinities(T, r):
    """A rank product beyond the largest float meets an infinity of its adapter: an infinity of the
    product's sign, and no NaN."""
    c = Case(T, 264, 4616, r, 4, "each", seed=5)
    c.of[T // 2] = 1
    t, l = T // 2, r - 3
    c.w[:, 0], c.w[0], c.x[:, 0], c.dy[:, 0] = 0, 0, 0, 0
    c.a[1, :, 0], c.b[1, 0] = 0, 0
    c.x[t, 0], c.a[1, l, 0] = 1e30, 1e20      # v[t, l] = inf
    c.dy[t, 0], c.b[1, 0, l] = 1e30, 1e20     # dv[t, l] = inf
    c.b[1, 5, l], c.b[1, 9, l] = float("inf"), -float("inf")
    c.a[1, l, 5], c.a[1, l, 9] = float("inf"), -float("inf")
    for z in (c.x, c.dy):                     # v[l] and dv[l] of all the adapter's tokens are inf, too
        z[:, 5], z[:, 9] = 1, -1
    y, v = c.forward()
    dx, _, _ = c.backward(v)
    mine = (c.of == 1).cuda()
    assert bool((v[mine][:, l] == float("inf")).all())
    for got in (y, dx):
        assert bool((got[mine][:, 5] == float("inf")).all()) and bool((got[mine][:, 9] == -float("inf")).all())
        assert bool(torch.isfinite(got[~mine].float()).all())


@pytest.mark.gpu
def test_gradients_against_differences():
    """The function is linear in x, in A (through v) and in B: f(z + h d) - f(z - h d) = 2 h <grad, d>.
    In fp64 from the definition with the kernel's gradients, each off by its tolerance."""
    c = Case(40, 72, 136, 16, 3, "each")
    _, v = c.forward()
    dx, da, db = (t.double().cpu() for t in c.backward(v))
    ref = c.reference()
    g = torch.Generator().manual_seed(2)

    def f(x, a, b):
        y = x @ c.w.double().t()
        for i in range(c.n):
            rows = torch.nonzero(c.of == i).flatten()
            y[rows] += float(c.s[i]) * (x[rows] @ a[i].t()) @ b[i].t()
        return float((y * c.dy.double()).sum())

    z = [c.x.double(), c.a.double(), c.b.double()]
    for k, (grad, name) in enumerate(((dx, "dx"), (da, "da"), (db, "db"))):
        d = torch.randn(z[k].shape, generator=g).double()
        h = 2.0 ** -10
        up, down = list(z), list(z)
        up[k], down[k] = z[k] + h * d, z[k] - h * d
        diff = (f(*up) - f(*down)) / (2 * h)
        tol = ((ref[name][1] + HALF * ref[name][0].abs()) * d.abs()).sum()
        assert abs(diff - float((grad * d).sum())) <= float(tol) + 1e-6 * abs(diff)


@pytest.mark.gpu
def test_out_of_range_ids_set_the_status_and_count_as_none():
    c = Case(40, 72, 136, 16, 3, "each")
    c.of[3], c.of[39] = 3, -2
    y, v = c.forward()
    assert m.moe_check_status() == m.MOE_ERR_DEVICE_STATUS
    c2 = Case(40, 72, 136, 16, 3, "each")
    c2.of = c.of.clone()
    c2.of[3], c2.of[39] = -1, -1
    y2, v2 = c2.forward()
    assert torch.equal(y, y2) and torch.equal(v, v2)
    g = c.backward(v)
    assert m.moe_check_status() == m.MOE_ERR_DEVICE_STATUS
    for s, t in zip(g, c2.backward(v2)):
        assert torch.equal(s, t)
    assert m.moe_check_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 300])
def test_repeats_bit_for_bit_from_a_graph_on_another_stream(T):
    c = Case(T, 1000, 616, 24, 5, "runs")
    t = {n: c.dev(getattr(c, n)) for n in ("x", "w", "a", "b", "s", "of", "dy")}
    y, v = c.forward()
    g = c.backward(v)
    out = [torch.empty_like(u) for u in (y, v, *g)]
    ws = scratch(c.p, T)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        m.moe_adapter_project(c.p, T, t["x"], t["w"], t["a"], t["b"], t["s"], t["of"], out[0], out[1], ws)
        m.moe_adapter_project_backward(c.p, T, t["dy"], t["x"], t["w"], t["a"], t["b"], t["s"], t["of"], out[1], out[2],
                                       out[3], out[4], ws)
    for _ in range(3):
        for o in out:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, (y, v, *g)))
    # other tokens and other requests in the captured buffers
    d = Case(T, 1000, 616, 24, 5, "each", seed=8)
    for n in ("x", "w", "a", "b", "s", "of", "dy"):
        t[n].copy_(getattr(d, n))
    graph.replay()
    torch.cuda.synchronize()
    y, v = d.forward()
    assert all(torch.equal(p, q) for p, q in zip(out, (y, v, *d.backward(v))))


# ------------------------------------------------------------------ refusals (no GPU)
def test_refusals():
    m.build_library()
    L = m.lib()
    b = ctypes.c_void_p(FAKE)
    mis = ctypes.c_void_p(FAKE + 8)
    inv = m.MOE_ERR_INVALID_ARG
    p = m.Adapter(512, 1024, 4, 16)
    need = m.moe_adapter_workspace_size(p, 40)
    assert need >= 40 * 16 * 2

    def fwd(p=p, T=40, x=b, w=b, a=b, bb=b, s=b, of=b, out=b, fp32=0, v=b, ws=b, n=1 << 40):
        return L.moe_adapter_project(ctypes.byref(p), T, x, w, a, bb, s, of, out, fp32, v, ws, n, None)

    def bwd(p=p, T=40, dy=b, x=b, w=b, a=b, bb=b, s=b, of=b, v=b, dx=b, da=b, db=b, ws=b, n=1 << 40):
        return L.moe_adapter_project_backward(ctypes.byref(p), T, dy, x, w, a, bb, s, of, v, dx, da, db, ws, n, None)

    for bad, code in ((m.Adapter(516, 1024, 4, 16), inv), (m.Adapter(512, 1028, 4, 16), inv),
                      (m.Adapter(512, 1024, 4, 12), inv), (m.Adapter(512, 1024, 0, 16), inv),
                      (m.Adapter(0, 1024, 4, 16), inv), (m.Adapter(512, -8, 4, 16), inv),
                      (m.Adapter(512, 1024, 4, 0), inv), (m.Adapter(512, 1024, 4, 264), m.MOE_ERR_UNSUPPORTED),
                      (m.Adapter(512, 1024, 4104, 16), m.MOE_ERR_UNSUPPORTED)):
        assert fwd(p=bad) == code and bwd(p=bad) == code and m.moe_adapter_workspace_size(bad, 40) == 0
    assert fwd(T=-1) == inv and bwd(T=-1) == inv and fwd(fp32=2) == inv
    for k in ("x", "w", "a", "bb", "of", "out"):
        assert fwd(**{k: None}) == inv, k
    for k in ("x", "w", "a", "bb", "out", "v", "ws"):
        assert fwd(**{k: mis}) == inv and "aligned" in m.last_error(), k
    for k in ("dy", "x", "w", "a", "bb", "of", "v", "da", "db"):
        assert bwd(**{k: None}) == inv, k
    for k in ("dy", "x", "w", "a", "bb", "v", "dx", "da", "db", "ws"):
        assert bwd(**{k: mis}) == inv, k
    assert fwd(n=need - 1) == m.MOE_ERR_WORKSPACE and bwd(n=need - 1) == m.MOE_ERR_WORKSPACE
    assert fwd(ws=None) == m.MOE_ERR_WORKSPACE and bwd(ws=None, n=0) == m.MOE_ERR_WORKSPACE
    # nothing to do
    assert fwd(T=0, x=None, out=None, ws=None, n=0) == m.MOE_OK
    assert bwd(T=0, da=None, db=None, dy=None) == m.MOE_OK
    assert bwd(dx=None, da=None, db=None) == m.MOE_OK
    assert L.moe_adapter_project(None, 4, b, b, b, b, b, b, b, 0, b, b, 1 << 40, None) == inv


def test_workspace_never_shrinks_as_the_batch_grows():
    for p in (m.Adapter(512, 1024, 4, 16), m.Adapter(7168, 2048, 64, 128), m.Adapter(2048, 7168, 1, 8)):
        sizes = [m.moe_adapter_workspace_size(p, T) for T in range(0, 3000)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_binding_checks_sizes_and_types():
    p = m.Adapter(16, 24, 2, 8)
    x = torch.zeros(3, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be"):
        m.moe_adapter_project(p, 3, x.float(), None, None, None, None, None, None)
    with pytest.raises(ValueError, match="x must be"):
        m.moe_adapter_project(p, 4, x, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="adapter_of"):
        m.moe_adapter_project(p, 3, None, None, None, None, None, torch.zeros(3, dtype=torch.int64), None)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_adapter_project(p, 3, x, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="out must be"):
        m.moe_adapter_project(p, 3, None, None, None, None, None, None, torch.zeros(3, 24, dtype=torch.float64))
