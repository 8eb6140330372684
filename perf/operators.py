"""The operators around the expert layer that `moe_expert_layer_06_gb300` adds, as cases with inputs, a plain form and the calls.

route          scored routing of T tokens from their router logits: sigmoid or softmax scores, a balance bias that acts on
               the selection only, expert groups, top-k, renormalised and scaled weights.
route_train    the same, then the gradient of the weights with respect to the logits.
adapter        a projection shared by all requests with each request's low-rank adapter beside it.
adapter_train  the same, then the gradients of its input and of every adapter (the shared weight is frozen).

`own` False: elementary torch operations; True: the package's entry points.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _route(name, T, E, k, score, groups=1, kept=1, top2=False, bias=True, renorm=True, scale=1.0, masked=False, train=False):
    return {"name": name, "op": "route_train" if train else "route", "T": T, "E": E, "k": k, "score": score, "groups": groups,
            "kept": kept, "top2": top2, "bias": bias, "renorm": renorm, "scale": scale, "masked": masked}


def _adapter(name, T, K, N, adapters, rank, runs, train=False):
    return {"name": name, "op": "adapter_train" if train else "adapter", "T": T, "K": K, "N": N, "adapters": adapters,
            "rank": rank, "runs": runs}


def listed():
    return [
        # one decoded token: 256 experts in 8 groups of which 4 are kept (latency)
        _route("route_t1", 1, 256, 8, "sigmoid", 8, 4, True, True, True, 2.5),
        # a ragged batch on a layer of 72 experts, some of them out of service
        _route("route_t1001_e72", 1001, 72, 6, "softmax", 1, 1, False, True, False, 1.0, True),
        # many experts, softmax over all of them, a bias that balances their loads
        _route("route_t8192_e1024", 8192, 1024, 8, "softmax", 1, 1, False, True, True, 1.0),
        # a long prompt batch
        _route("route_t65536", 65536, 256, 8, "sigmoid", 8, 4, True, True, True, 2.5),
        # training: forward and gradient, sigmoid scores (only the selected logits have one)
        _route("route_train_t4096", 4096, 256, 8, "sigmoid", 8, 4, True, True, True, 2.5, False, True),
        # training: softmax weights as they are (every logit has a gradient)
        _route("route_train_t16384", 16384, 256, 8, "softmax", 8, 3, False, False, False, 1.0, False, True),
        # one decoded token with its adapter, on the gate projection of a shared expert (latency)
        _adapter("adapter_t1", 1, 7168, 2048, 8, 16, False),
        # a decode batch, nearly every request with an adapter of its own
        _adapter("adapter_t32", 32, 7168, 2048, 64, 16, False),
        # a larger decode batch on the down projection of a shared expert
        _adapter("adapter_t192", 192, 2048, 7168, 24, 32, False),
        # a prompt batch of several requests on the stacked projection of two shared experts
        _adapter("adapter_t4096", 4096, 7168, 4096, 16, 64, True),
        # training a few adapters on ragged sizes
        _adapter("adapter_train_t777", 777, 1000, 616, 3, 24, True, True),
        # training adapters of the gate projection
        _adapter("adapter_train_t4096", 4096, 7168, 2048, 4, 64, True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        train = rng.random() < 0.4
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.choice([4, 6, 8, 9, 16, 18, 32, 40, 64, 128] if groups > 1 else [8, 60, 64, 72, 128, 160, 250, 256, 384, 512, 1000, 1024])
        E = min(1024, groups * per)
        groups = 1 if E != groups * per else groups
        kept = rng.randint(1, groups)
        k = rng.randint(2 if train else 1, min(8, kept * (E // groups)))
        most = min(65536, 65536 * 256 // E) // (4 if train else 1)
        score = rng.choice(["sigmoid", "softmax"])
        return {"op": "route_train" if train else "route", "T": _log(rng, 1, most), "E": E, "k": k, "score": score, "groups": groups,
                "kept": kept, "top2": groups > 1 and rng.random() < 0.5, "bias": rng.random() < 0.6, "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.random() < 0.25}
    train = rng.random() < 0.4
    K, N = 8 * _log(rng, 24, 1024), 8 * _log(rng, 24, 1024)
    most = int(min(4096, (4096 * 7168 * 2048 if train else 4096 * 7168 * 4096) // (K * N)))
    runs = train or rng.random() < 0.5
    T = _log(rng, 16 if train else 1, most if runs else min(most, 256))
    return {"op": "adapter_train" if train else "adapter", "T": T, "K": K, "N": N, "adapters": _log(rng, 1, 16 if runs else 64),
            "rank": 8 * _log(rng, 1, 16 if T <= 1024 else 8), "runs": runs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T = case["T"]
    s = dict(case)
    if case["op"].startswith("route"):
        E, k = case["E"], case["k"]
        # logits of a linear router with weights of deviation 0.02 on unit activations of width 7168
        s["logits"] = torch.randn(T, E, device=DEV, generator=g) * 1.69
        if case["masked"]:
            # experts out of service have the logit -inf (at least k, and one of every group, remain)
            off = torch.arange(E, device=DEV) % 16 == 1 + seed % 3
            off &= torch.arange(E, device=DEV) % max(1, E // case["groups"]) != 0
            if E - int(off.sum()) >= 2 * k and case["groups"] == 1:
                s["logits"][:, off] = -math.inf
        s["b"] = torch.randn(E, device=DEV, generator=g) * 0.05 if case["bias"] else None
        s["dw"] = torch.randn(T, k, device=DEV, generator=g) if case["op"] == "route_train" else None
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["w"] = torch.empty(T, k, device=DEV)
        s["dlogits"] = torch.empty(T, E, device=DEV) if case["op"] == "route_train" else None
        return s
    K, N, nA, r = case["K"], case["N"], case["adapters"], case["rank"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device=DEV, generator=g) * std).to(torch.bfloat16)

    s["x"] = normal(T, K)
    s["weight"] = normal(N, K, std=K ** -0.5)
    s["a"] = normal(nA, r, K, std=K ** -0.5)
    s["bb"] = normal(nA, N, r, std=0.5 * r ** -0.5)
    s["scaling"] = torch.rand(nA, device=DEV, generator=g) * 1.5 + 0.5
    # requests: one token each, or a run of consecutive tokens; one in eight after the first has no adapter (-1)
    rs = np.random.RandomState(seed % (1 << 31))
    if case["runs"]:
        cuts = np.sort(rs.randint(0, T + 1, max(0, T // 256)))
        lengths = np.diff(np.concatenate([[0], cuts, [T]]))
    else:
        lengths = np.ones(T, dtype=np.int64)
    of = rs.randint(0, nA, len(lengths))
    of[1:][rs.randint(0, 8, len(lengths) - 1) == 0] = -1
    s["of"] = torch.from_numpy(np.repeat(of, lengths).astype(np.int32)).to(DEV)
    s["y"] = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    if case["op"] == "adapter_train":
        s["dy"] = normal(T, N)
        s["v"] = torch.empty(T, r, dtype=torch.bfloat16, device=DEV)
        s["dx"] = torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
        s["da"] = torch.empty(nA, r, K, dtype=torch.bfloat16, device=DEV)
        s["db"] = torch.empty(nA, N, r, dtype=torch.bfloat16, device=DEV)
    return s


def work(case):
    T = case["T"]
    if case["op"].startswith("route"):
        E, k = case["E"], case["k"]
        nbytes, flops = T * E * 4 + T * k * 8 + (E * 4 if case["bias"] else 0), 10 * T * E
        if case["op"] == "route_train":
            nbytes += T * k * 4 + T * E * 4
            flops += 4 * T * E if case["score"] == "softmax" and not case["renorm"] else 0
        return {"bytes": nbytes, "flops": flops}
    K, N, r = case["K"], case["N"], case["rank"]
    used = min(case["adapters"], T // 256 + 1 if case["runs"] else T)
    nbytes = 2 * (N * K + T * (K + N) + used * r * (K + N)) + T * 4
    flops = 2 * T * K * N + 2 * T * r * (K + N)
    if case["op"] == "adapter_train":
        nbytes += 2 * (T * (K + N) + case["adapters"] * r * (K + N))
        flops += 2 * T * K * N + 4 * T * r * (K + N)
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    if state["op"].startswith("route"):
        return _plain_route(state)
    return _plain_adapter(state)


def _run_own(s):
    import moe_expert_layer_06_gb300 as m
    T = s["T"]
    if s["op"].startswith("route"):
        if "shape" not in s:
            s["shape"] = m.Shape(8, 8, s["E"], s["k"], 0, 0, s["E"], 1)
            s["router"] = m.Router(m.MOE_SCORE_SIGMOID if s["score"] == "sigmoid" else m.MOE_SCORE_SOFTMAX, s["groups"], s["kept"],
                                   m.MOE_GROUP_TOP2 if s["top2"] else m.MOE_GROUP_MAX, int(s["renorm"]), s["scale"])
        m.moe_route_scored(s["shape"], s["router"], T, None, None, s["b"], s["logits"], None, s["idx"], s["w"])
        if s["op"] == "route":
            return s["idx"], s["w"]
        m.moe_route_scored_backward(s["shape"], s["router"], T, s["logits"], s["idx"], s["dw"], s["dlogits"])
        return s["idx"], s["w"], s["dlogits"]
    if "adapter" not in s:
        s["adapter"] = m.Adapter(s["K"], s["N"], s["adapters"], s["rank"])
        s["ws"] = torch.empty(m.moe_adapter_workspace_size(s["adapter"], T), dtype=torch.uint8, device=DEV)
    m.moe_adapter_project(s["adapter"], T, s["x"], s["weight"], s["a"], s["bb"], s["scaling"], s["of"], s["y"], s.get("v"), s["ws"])
    if s["op"] == "adapter":
        return s["y"]
    m.moe_adapter_project_backward(s["adapter"], T, s["dy"], s["x"], s["weight"], s["a"], s["bb"], s["scaling"], s["of"], s["v"],
                                   s["dx"], s["da"], s["db"], s["ws"])
    return s["y"], s["dx"], s["da"], s["db"]


def _plain_route(s):
    l, T, E, k, G = s["logits"], s["T"], s["E"], s["k"], s["groups"]
    # the selection compares values next to one another: 64 bits
    d = l.double()
    c = torch.sigmoid(d) if s["score"] == "sigmoid" else torch.softmax(d, 1)
    if s["b"] is not None:
        c = c + s["b"].double()
    c = torch.where(d == -math.inf, d, c)
    if s["kept"] < G:
        per = c.view(T, G, E // G)
        gs = per.sort(dim=2, descending=True).values
        second = gs[:, :, 1] if s["top2"] and E // G > 1 else torch.zeros_like(gs[:, :, 0])
        gs = gs[:, :, 0] + torch.where(second == -math.inf, 0.0, second)  # a masked second best counts nothing
        best = gs.sort(dim=1, descending=True, stable=True).indices[:, :s["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, best, True)
        c = per.masked_fill(~keep[:, :, None], -math.inf).view(T, E)
    idx = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    lk = l.gather(1, idx)
    # s_j over a common factor: exp of the logit's negative part relative to the row's largest
    if s["score"] == "sigmoid":
        score = torch.sigmoid(lk)
        rest = torch.sigmoid(-lk)
        low = lk.clamp(max=0.0)
        share = torch.exp(low - low.amax(1, keepdim=True)) / (1.0 + torch.exp(-lk.abs()))
    else:
        p = torch.softmax(l, 1)
        score = p.gather(1, idx)
        rest = None
        share = torch.exp(lk - lk.amax(1, keepdim=True))
    share = share / share.sum(1, keepdim=True)
    w = (share if s["renorm"] else score) * s["scale"]
    if s["op"] == "route":
        return idx.to(torch.int32), w
    dw = s["dw"]
    if s["renorm"]:
        dl = s["scale"] * share * (dw - (share * dw).sum(1, keepdim=True))
        if rest is not None:
            dl = dl * rest
        full = torch.zeros_like(l).scatter_(1, idx, dl)
    elif rest is not None:
        full = torch.zeros_like(l).scatter_(1, idx, s["scale"] * dw * score * rest)
    else:
        ds = torch.zeros_like(l).scatter_(1, idx, s["scale"] * dw)
        full = p * (ds - (ds * p).sum(1, keepdim=True))
    return idx.to(torch.int32), w, full


def _plain_adapter(s):
    x, weight = s["x"].float(), s["weight"].float()
    nA, r, K, N, T = s["adapters"], s["rank"], s["K"], s["N"], s["T"]
    a, b = s["a"].float().view(nA * r, K), s["bb"].float()
    # every adapter on every row, and each row keeps its own
    factor = torch.where(s["of"][:, None] == torch.arange(nA, device=x.device), s["scaling"][None, :], 0.0)
    v = ((x @ a.t()).view(T, nA, r) * factor[:, :, None]).view(T, nA * r)
    y = x @ weight.t() + v @ b.transpose(1, 2).reshape(nA * r, N)
    if s["op"] == "adapter":
        return y.to(torch.bfloat16)
    dy = s["dy"].float()
    dv = ((dy @ b.transpose(0, 1).reshape(N, nA * r)).view(T, nA, r) * factor[:, :, None]).view(T, nA * r)
    dx = dy @ weight + dv @ a
    da = (dv.t() @ x).view(nA, r, K)
    db = (dy.t() @ v).view(N, nA, r).transpose(0, 1).contiguous()
    return tuple(t.to(torch.bfloat16) for t in (y, dx, da, db))


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("route"):
        return _exact_route(s)
    x, weight, a, b = (s[n].double() for n in ("x", "weight", "a", "bb"))
    y = torch.matmul(x, weight.T)
    train = case["op"] == "adapter_train"
    if train:
        dy = s["dy"].double()
        dx, da, db = torch.matmul(dy, weight), torch.zeros_like(a), torch.zeros_like(b)
    for i in range(case["adapters"]):
        rows = torch.nonzero(s["of"] == i).flatten()
        if rows.numel() == 0:
            continue
        f = float(s["scaling"][i])
        v = x[rows] @ a[i].T * f
        y[rows] += v @ b[i].T
        if train:
            dv = dy[rows] @ b[i] * f
            dx[rows] += dv @ a[i]
            da[i] = dv.T @ x[rows]
            db[i] = dy[rows].T @ v
    return (y, dx, da, db) if train else y


def _exact_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    l = s["logits"].double().requires_grad_(s["op"] == "route_train")
    d = l.detach()
    masked = d == -math.inf
    score = 1.0 / (1.0 + torch.exp(-l)) if s["score"] == "sigmoid" else torch.softmax(l, 1)
    c = score.detach() + (s["b"].double() if s["b"] is not None else 0.0)
    c = c.masked_fill(masked, -math.inf)
    ids = torch.arange(E, device=d.device)

    def first_best(v, n):
        """Columns of the n best values of each row, one after the other, equal values by the lower column."""
        v, cols = v.clone(), torch.arange(v.shape[1], device=v.device)
        taken = torch.zeros_like(v, dtype=torch.bool)
        out = []
        for _ in range(n):
            top = v.masked_fill(taken, -math.inf).amax(1, keepdim=True)
            at = torch.where((v == top) & ~taken, cols, v.shape[1]).amin(1, keepdim=True)
            taken.scatter_(1, at, True)
            out.append(at)
        return torch.cat(out, 1)

    allowed = torch.ones(T, E, dtype=torch.bool, device=d.device)
    if s["kept"] < G:
        per = c.view(T, G, -1)
        of_group = per.amax(2)
        if s["top2"] and E // G > 1:
            second = per.topk(2, 2).values[:, :, 1]
            of_group = of_group + second.masked_fill(second == -math.inf, 0.0)
        groups = first_best(of_group, s["kept"])
        allowed = ((ids // (E // G))[None, :, None] == groups[:, None, :]).any(2)
    idx = first_best(c.masked_fill(~allowed, -math.inf), k)
    w = score.gather(1, idx)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * s["scale"]
    if s["op"] == "route":
        return idx.to(torch.int32), w
    w.backward(s["dw"].double())
    return idx.to(torch.int32), w.detach(), l.grad
