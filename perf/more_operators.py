"""The operators that train the expert layer of `moe_expert_layer_06_gb300`, as cases with inputs, a plain form and the calls.

project       matrix products grouped by expert: the rows of each expert's slot (ragged counts) times its weights, one part
              or two (gate and up) side by side.
project_grad  their gradients: of the rows and of every expert's weights; the rows in bf16, or kept in 8 bits.
keep          rows kept in 8 bits for the backward pass: E4M3 codes and a power of two for each 128 columns.
swiglu        SwiGLU whose gate and up are kept in 8 bits, then its gradient from what was kept, with the activation again.
combine_grad  the gradient of the combine: of every expert output row and of the routing weights.

`own` False: elementary torch operations; True: the package's entry points.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
BLOCK = 128  # columns that share a scale


# ------------------------------------------------------------------ cases
def _project(name, rows, K, N, slots, parts, skew, grad=False, eight=False):
    return {"name": name, "op": "project_grad" if grad else "project", "rows": rows, "K": K, "N": N, "slots": slots, "parts": parts,
            "skew": skew, "eight": eight}


def listed():
    return [
        # gate and up of a small layer, ragged in every size (latency)
        _project("project_r400", 400, 600, 328, 16, 2, 0.5),
        # gate and up of 32 experts, 512 tokens to 8 of them each: as many weights as rows can use
        _project("project_r4096", 4096, 7168, 2048, 32, 2, 0.3),
        # the same for a batch of 4096 tokens
        _project("project_r32768", 32768, 7168, 2048, 32, 2, 0.3),
        # gradients of a small down projection, some experts without a row (latency)
        _project("grad_r100", 100, 328, 600, 16, 1, 1.0, True),
        # gradients of the down projections of 32 experts
        _project("grad_r4096", 4096, 2048, 7168, 32, 1, 0.3, True),
        # gradients of gate and up, a batch of 4096 tokens whose dispatched rows were kept in 8 bits
        _project("grad8_r32768", 32768, 7168, 2048, 32, 2, 0.3, True, True),
        # a ragged batch of rows to keep
        {"name": "keep_r1001", "op": "keep", "rows": 1001, "cols": 600},
        # the dispatched rows of 4096 tokens
        {"name": "keep_r32768", "op": "keep", "rows": 32768, "cols": 7168},
        # the rows of one token (latency)
        {"name": "swiglu_r8", "op": "swiglu", "rows": 8, "inter": 2048},
        # the rows of 4096 tokens
        {"name": "swiglu_r32768", "op": "swiglu", "rows": 32768, "inter": 2048},
        # a small layer's batch (latency)
        {"name": "combine_t100", "op": "combine_grad", "T": 100, "k": 4, "hidden": 600},
        # a batch of 4096 tokens
        {"name": "combine_t4096", "op": "combine_grad", "T": 4096, "k": 8, "hidden": 7168},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["project", "project", "project_grad", "project_grad", "keep", "swiglu", "combine_grad"])
    if kind.startswith("project"):
        grad = kind == "project_grad"
        eight = grad and rng.random() < 0.5
        K, N = 16 * _log(rng, 4, 448), 8 * _log(rng, 8, 896)
        parts = rng.choice([1, 2])
        K = K if eight or rng.random() < 0.5 else K - 8
        slots = _log(rng, 1, max(1, min(256, 32 * 7168 * 4096 // (K * N * parts))))
        rows = _log(rng, 1, min(32768, 32768 * 7168 * 4096 // (K * N * parts)))
        return {"op": kind, "rows": rows, "K": K, "N": N, "slots": slots, "parts": parts, "skew": rng.choice([0.0, 0.3, 1.0]), "eight": eight}
    if kind == "keep":
        cols = 8 * _log(rng, 1, 1024)
        return {"op": kind, "rows": _log(rng, 1, min(65536, 32768 * 7168 // cols)), "cols": cols}
    if kind == "swiglu":
        inter = 8 * _log(rng, 1, 1024)
        return {"op": kind, "rows": _log(rng, 1, min(65536, 32768 * 2048 // inter)), "inter": inter}
    k, hidden = rng.randint(1, 10), 8 * _log(rng, 1, 1024)
    return {"op": kind, "T": _log(rng, 1, min(16384, 4096 * 8 * 7168 // (k * hidden))), "k": k, "hidden": hidden}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device=DEV, generator=g) * std).to(torch.bfloat16)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=DEV)

    def activations(rows, cols):
        # columns of different sizes, and now and then a value far above the others
        std = torch.exp(0.5 * torch.randn(cols, device=DEV, generator=g))
        v = torch.randn(rows, cols, device=DEV, generator=g) * std
        return torch.where(torch.rand(rows, cols, device=DEV, generator=g) < 1e-3, v * 12.0, v).to(torch.bfloat16)

    if case["op"] == "keep":
        s["x"] = activations(case["rows"], case["cols"])
        s["codes"] = empty(case["rows"], case["cols"], dtype=torch.uint8)
        s["scale"] = empty(case["rows"], -(-case["cols"] // BLOCK), dtype=torch.float32)
        return s
    if case["op"] == "swiglu":
        R, I = case["rows"], case["inter"]
        s["gate_up"] = activations(R, 2 * I)
        s["dh"] = normal(R, I, std=0.1)
        s["h"], s["h_again"], s["d_gate_up"] = empty(R, I), empty(R, I), empty(R, 2 * I)
        s["codes"] = empty(R, 2 * I, dtype=torch.uint8)
        s["scale"] = empty(R, 2 * -(-I // BLOCK), dtype=torch.float32)
        return s
    if case["op"] == "combine_grad":
        T, k, H = case["T"], case["k"], case["hidden"]
        s["dout"], s["y"] = normal(T, H, std=0.1), normal(T * k, H)
        s["w"] = torch.softmax(torch.randn(T, k, device=DEV, generator=g), 1)
        s["inv_perm"] = torch.randperm(T * k, device=DEV, generator=g).to(torch.int32)
        s["dy"], s["dw"] = empty(T * k, H), empty(T, k, dtype=torch.float32)
        return s
    R, K, N, S, P = (case[n] for n in ("rows", "K", "N", "slots", "parts"))
    rs = np.random.RandomState(seed % (1 << 31))
    p = np.exp(case["skew"] * rs.randn(S))
    counts = rs.multinomial(R, p / p.sum())
    s["counts"], s["most"] = counts, int(counts.max())
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
    s["weights"] = [normal(S, N, K, std=K ** -0.5) for _ in range(P)]
    if case["op"] == "project":
        s["x"] = normal(R, K)
        s["y"] = empty(R, P * N)
        return s
    s["dy"] = normal(R, P * N, std=0.1)
    if case["eight"]:
        x = activations(R, K)
        codes, s["x8_scale"] = _keep(x)
        s["x8"] = codes.view(torch.uint8)
    else:
        s["x"] = normal(R, K)
    s["dx"] = empty(R, K)
    s["dweights"] = [empty(S, N, K) for _ in range(P)]
    return s


def work(case):
    if case["op"] == "keep":
        n, b = case["rows"] * case["cols"], case["rows"] * -(-case["cols"] // BLOCK)
        return {"bytes": 3 * n + 4 * b, "flops": 3 * n}
    if case["op"] == "swiglu":
        n, b = case["rows"] * case["inter"], 2 * case["rows"] * -(-case["inter"] // BLOCK)
        return {"bytes": (4 + 2 + 2) * n + 4 * b + (2 + 2 + 4 + 2) * n + 4 * b, "flops": 40 * n}
    if case["op"] == "combine_grad":
        T, k, H = case["T"], case["k"], case["hidden"]
        return {"bytes": 2 * T * H + 4 * T * k * H + 12 * T * k, "flops": 3 * T * k * H}
    R, K, N, S, P = (case[n] for n in ("rows", "K", "N", "slots", "parts"))
    used = S * (1.0 - (1.0 - 1.0 / S) ** R)  # experts with a row
    if case["op"] == "project":
        return {"bytes": 2 * (used * P * N * K + R * (K + P * N)), "flops": 2 * R * K * N * P}
    return {"bytes": 2 * (used * P * N * K + S * P * N * K + R * (K + P * N)) + R * K * (1 if case["eight"] else 2), "flops": 4 * R * K * N * P}


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def _run_own(s):
    import moe_expert_layer_06_gb300 as m
    if s["op"] == "keep":
        m.moe_checkpoint_rows(s["rows"], s["cols"], s["x"], s["codes"], s["scale"])
        return s["codes"].view(torch.float8_e4m3fn), s["scale"]
    if s["op"] == "swiglu":
        R, I = s["rows"], s["inter"]
        m.moe_swiglu_checkpoint(R, I, s["gate_up"], s["h"], s["codes"], s["scale"])
        m.moe_swiglu_backward(R, I, s["codes"], s["scale"], s["dh"], s["d_gate_up"], s["h_again"])
        return s["h"], s["codes"].view(torch.float8_e4m3fn), s["scale"], s["d_gate_up"], s["h_again"]
    if s["op"] == "combine_grad":
        if "shape" not in s:
            s["shape"] = m.Shape(s["hidden"], 8, s["k"], s["k"], 0, 0, s["k"], 1)
        m.moe_combine_backward(s["shape"], s["T"], s["dout"], s["y"], s["inv_perm"], s["w"], s["dy"], s["dw"])
        return s["dy"], s["dw"]
    if "project" not in s:
        s["project"] = m.Project(s["K"], s["N"], s["slots"], s["parts"])
    w, w2 = (s["weights"] + [None])[:2]
    if s["op"] == "project":
        m.moe_expert_project(s["project"], s["rows"], s["x"], s["offsets"], w, w2, s["y"])
        return s["y"]
    dw, dw2 = (s["dweights"] + [None])[:2]
    m.moe_expert_project_backward(s["project"], s["rows"], s["dy"], s.get("x"), s.get("x8"), s.get("x8_scale"), s["offsets"], w, w2,
                                  s["dx"], dw, dw2)
    return s["dx"], s["dweights"]


# ------------------------------------------------------------------ the plain forms
def _keep(x):
    """Codes and scales of rows: the least power of two (2^-117 at least) that brings a block's largest value to 448 at most."""
    R, C = x.shape
    nb = -(-C // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - C)).view(R, nb, BLOCK)
    m, e = torch.frexp(v.abs().amax(2))
    e = torch.where(m == 0.0, 0, (e - torch.where(m > 0.875, 8, 9)).clamp(min=-117))
    scale = ((e + 127) << 23).to(torch.int32).view(torch.float32)  # (pow(2, e) may be a step off)
    codes = (v / scale[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(R, nb * BLOCK)[:, :C].contiguous(), scale


def _kept(codes, scale):
    C = codes.shape[1]
    return codes.float() * scale.repeat_interleave(BLOCK, 1)[:, :C]


def _plain_keep(s):
    return _keep(s["x"])


def _plain_swiglu(s):
    gate, up = s["gate_up"].float().chunk(2, 1)
    h = gate * torch.sigmoid(gate) * up
    kg, ku = _keep(s["gate_up"][:, :s["inter"]]), _keep(s["gate_up"][:, s["inter"]:])
    g, u, dh = _kept(*kg), _kept(*ku), s["dh"].float()
    sg = torch.sigmoid(g)
    dgu = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], 1)
    bf16 = torch.bfloat16
    codes = torch.cat([kg[0].view(torch.uint8), ku[0].view(torch.uint8)], 1).view(torch.float8_e4m3fn)
    return h.to(bf16), codes, torch.cat([kg[1], ku[1]], 1), dgu.to(bf16), (g * sg * u).to(bf16)


def _plain_combine_grad(s):
    T, k, H = s["T"], s["k"], s["hidden"]
    row = s["inv_perm"].long()
    d = s["dout"].float()[:, None, :]
    dw = (s["y"][row].float().view(T, k, H) * d).sum(2)
    dy = torch.empty_like(s["y"])
    dy[row] = (s["w"][:, :, None] * d).view(T * k, H).to(torch.bfloat16)
    return dy, dw


def _padded(s):
    """[slots, most]: the row of each place of each slot (row 0 past its end), and whether there is one."""
    start, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = start[:, None] + torch.arange(s["most"], device=DEV)[None, :]
    there = at < end[:, None]
    return torch.where(there, at, 0), there


def _plain_project(s):
    at, there = _padded(s)
    x = s["x"].float()[at]
    y = torch.cat([torch.bmm(x, w.float().transpose(1, 2)) for w in s["weights"]], 2)
    out = torch.empty(s["rows"], y.shape[2], dtype=torch.bfloat16, device=DEV)
    out[at[there]] = y[there].to(torch.bfloat16)
    return out


def _plain_project_grad(s):
    at, there = _padded(s)
    x = _kept(s["x8"].view(torch.float8_e4m3fn), s["x8_scale"]) if s["eight"] else s["x"].float()
    x = x[at] * there[:, :, None]
    dy = s["dy"].float()[at] * there[:, :, None]
    dys = dy.split(s["N"], 2)
    dx = torch.bmm(dys[0], s["weights"][0].float())
    if s["parts"] == 2:
        dx = dx + torch.bmm(dys[1], s["weights"][1].float())
    out = torch.empty(s["rows"], s["K"], dtype=torch.bfloat16, device=DEV)
    out[at[there]] = dx[there].to(torch.bfloat16)
    return out, [torch.bmm(d.transpose(1, 2), x).to(torch.bfloat16) for d in dys]


_PLAIN = {"keep": _plain_keep, "swiglu": _plain_swiglu, "combine_grad": _plain_combine_grad, "project": _plain_project,
          "project_grad": _plain_project_grad}


# ------------------------------------------------------------------ in 64 bits
def _exponent(v):
    """floor(log2(v)) of positive numbers of 64 bits, and a large negative one of 0 (log2 itself may be a step off)."""
    return ((v.view(torch.int64) >> 52) & 0x7FF) - 1023


def _two_to(e):
    return ((e + 1023) << 52).view(torch.float64)


def _exact_keep(x):
    """Values of the codes, and the scales, in 64 bits."""
    R, C = x.shape
    codes, scales = torch.zeros(R, C, dtype=torch.float64, device=DEV), []
    for c in range(0, C, BLOCK):
        v = x[:, c:c + BLOCK].double()
        top = v.abs().amax(1, keepdim=True)
        e = _exponent(top)
        e = torch.where(top > 1.75 * _two_to(e), e + 1, e) - 8  # 448 is 1.75 * 2^8
        scale = torch.where(top == 0.0, 1.0, _two_to(e.clamp(min=-117)))
        v = v / scale
        step = _two_to(_exponent(v.abs()).clamp(min=-6) - 3)
        codes[:, c:c + BLOCK] = torch.round(v / step) * step
        scales.append(scale)
    return codes, torch.cat(scales, 1)


def _exact_values(codes, scale):
    out = codes.clone()
    for b in range(scale.shape[1]):
        out[:, b * BLOCK:(b + 1) * BLOCK] *= scale[:, b:b + 1]
    return out


def _exact_swiglu(s):
    I = s["inter"]
    gate, up = s["gate_up"][:, :I].double(), s["gate_up"][:, I:].double()
    h = gate / (1.0 + torch.exp(-gate)) * up
    cg, sg = _exact_keep(s["gate_up"][:, :I])
    cu, su = _exact_keep(s["gate_up"][:, I:])
    g, u = _exact_values(cg, sg).requires_grad_(True), _exact_values(cu, su).requires_grad_(True)
    again = g / (1.0 + torch.exp(-g)) * u
    again.backward(s["dh"].double())
    return h, torch.cat([cg, cu], 1), torch.cat([sg, su], 1), torch.cat([g.grad, u.grad], 1), again.detach()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "keep":
        return _exact_keep(s["x"])
    if case["op"] == "swiglu":
        return _exact_swiglu(s)
    if case["op"] == "combine_grad":
        T, k, H = case["T"], case["k"], case["hidden"]
        dy, dw = torch.zeros(T * k, H, dtype=torch.float64, device=DEV), torch.zeros(T, k, dtype=torch.float64, device=DEV)
        d = s["dout"].double()
        for j in range(k):
            row = s["inv_perm"].view(T, k)[:, j].long()
            dw[:, j] = torch.einsum("th,th->t", s["y"][row].double(), d)
            dy[row] = s["w"][:, j:j + 1].double() * d
        return dy, dw
    R, K, N, P = (case[n] for n in ("rows", "K", "N", "parts"))
    grad = case["op"] == "project_grad"
    if grad:
        x = _exact_values(s["x8"].view(torch.float8_e4m3fn).double(), s["x8_scale"].double()) if case["eight"] else s["x"].double()
        dx = torch.zeros(R, K, dtype=torch.float64, device=DEV)
        dw = [torch.zeros(w.shape, dtype=torch.float64, device=DEV) for w in s["weights"]]
    else:
        x = s["x"].double()
        y = torch.zeros(R, P * N, dtype=torch.float64, device=DEV)
    end = np.cumsum(s["counts"])
    for e in np.nonzero(s["counts"])[0]:
        rows = slice(int(end[e] - s["counts"][e]), int(end[e]))
        for p in range(P):
            w = s["weights"][p][e].double()
            cols = slice(p * N, (p + 1) * N)
            if grad:
                dy = s["dy"][rows, cols].double()
                dx[rows] += dy @ w
                dw[p][e] = dy.T @ x[rows]
            else:
                y[rows, cols] = x[rows] @ w.T
    return (dx, dw) if grad else y
