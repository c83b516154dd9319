"""The training-step operators that work on a plan's flat buffers, as measurable cases.

Four operators: an embedding lookup straight from a gathered flat buffer, its
gradient straight into the packed flat buffer, the orthogonalisation of whole
matrices by Newton-Schulz products, and the Muon step built on it. Each case
says how large; ``run`` computes it in plain torch operations, or, where
``own`` is true, by this package's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
COEFFS = (3.4445, -4.7750, 2.0315)      # the quintic of the published Muon optimiser
STEPS = 5
EPS = 1e-7
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ALIGN = 16


class Spec:
    """One tensor of a group, with the fields the planner reads."""

    def __init__(self, name, rows, cols, kind, p0=0, p1=0):
        self.name, self.rows, self.cols, self.kind, self.p0, self.p1 = name, rows, cols, kind, p0, p1


def listed():
    return [
        # the smallest matrix of the repository's tiny group: latency alone
        {"name": "ortho 64x48 f32", "op": "ortho", "shapes": "64x48", "dt": "f32"},
        # one key projection of a Llama-3-8B layer, from a bf16 reduce-scatter
        {"name": "ortho 1024x4096 bf16", "op": "ortho", "shapes": "1024x4096", "dt": "bf16"},
        # two experts of the 2880-wide MoE layer, one matrix tall and one square
        {"name": "ortho moe 2 experts", "op": "ortho", "shapes": "5760x2880,2880x2880,5760x2880,2880x2880", "dt": "f32"},
        # the router of the MoE layer, and an odd matrix, as a group of small ones
        {"name": "muon router", "op": "muon", "shapes": "128x2880,333x1001", "dt": "f32", "lr": 1e-4, "wd": 0.1, "nesterov": True},
        # all seven matrices of a Llama-3-8B layer in one step
        {"name": "muon 8b layer", "op": "muon", "shapes": "4096x4096,1024x4096,1024x4096,4096x4096,14336x4096,14336x4096,4096x14336", "dt": "f32", "lr": 1e-4, "wd": 0.1, "nesterov": True},
        # the widest matrix of a Llama-3-70B layer on the rank that holds it whole
        {"name": "muon 8192x28672", "op": "muon", "shapes": "8192x28672", "dt": "bf16", "lr": 1e-4, "wd": 0.1, "nesterov": False},
        # one token, as a server's single step looks it up
        {"name": "embed 1 token", "op": "embed", "rows": 131072, "cols": 4096, "tokens": 1, "dt": "bf16", "out": "bf16", "scale": 64.0, "idx": "i64"},
        # a training micro-batch of two 8192-token sequences
        {"name": "embed 16384 tokens", "op": "embed", "rows": 131072, "cols": 8192, "tokens": 16384, "dt": "bf16", "out": "bf16", "scale": 1.0, "idx": "i64"},
        # an odd width out of an fp32 buffer, for a batch that is not full
        {"name": "embed 4097 odd", "op": "embed", "rows": 32001, "cols": 1001, "tokens": 4097, "dt": "f32", "out": "bf16", "scale": 31.6, "idx": "i32"},
        # tied embeddings: the head's gradient is packed already, a few tokens are added to it
        {"name": "embed grad 512 tied", "op": "embed_grad", "rows": 50000, "cols": 2880, "tokens": 512, "dt": "bf16", "packed": "f32", "mode": "add", "scale": 1.0, "idx": "i64"},
        # a training micro-batch, the whole table's gradient written
        {"name": "embed grad 16384", "op": "embed_grad", "rows": 131072, "cols": 4096, "tokens": 16384, "dt": "bf16", "packed": "f32", "mode": "write", "scale": 64.0, "idx": "i64"},
        # fp32 gradients of an odd width, packed for a bf16 reduce-scatter
        {"name": "embed grad 4097 odd", "op": "embed_grad", "rows": 32001, "cols": 1001, "tokens": 4097, "dt": "f32", "packed": "bf16", "mode": "write", "scale": 31.6, "idx": "i32"},
    ]


def _log(rng, lo, hi):
    """A whole number spread over its logarithm, ends included, odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("ortho", "muon", "embed", "embed_grad"))
    if op in ("ortho", "muon"):
        # mostly one side near a model's width and the other up to four times it
        shapes, cost = [], 0.0
        for _ in range(rng.randint(1, 4)):
            a = _log(rng, 8, 5000)
            b = _log(rng, max(1, a // 4), min(4 * a, 15000))
            if rng.random() < 0.5:
                a, b = max(16, a // 16 * 16), max(16, b // 16 * 16)
            m, n = min(a, b), max(a, b)
            c = STEPS * (3.0 * m * m * n + m ** 3)
            if cost + c <= 1.2e13 and (not shapes or f"{a}x{b}" not in shapes):
                shapes.append(f"{a}x{b}")
                cost += c
        case = {"op": op, "shapes": ",".join(shapes or ["257x513"]), "dt": rng.choice(("f32", "bf16"))}
        if op == "muon":
            case.update(lr=round(math.exp(rng.uniform(math.log(2e-5), math.log(2e-4))), 7), wd=rng.choice((0.0, 0.1)),
                        nesterov=rng.random() < 0.7)
        return case
    rows, cols = _log(rng, 1000, 131072), _log(rng, 64, 8192)
    if rng.random() < 0.6:
        cols = max(64, cols // 64 * 64)
    rows = min(rows, (1 << 29) // cols)
    tokens = min(_log(rng, 1, 65536), (1 << 27) // cols)
    case = {"op": op, "rows": rows, "cols": cols, "tokens": tokens, "dt": rng.choice(("f32", "bf16")),
            "scale": rng.choice((1.0, round(math.sqrt(cols), 3))), "idx": rng.choice(("i64", "i32"))}
    if op == "embed":
        case["out"] = rng.choice(("f32", "bf16"))
    else:
        case["mode"] = rng.choice(("write", "add"))
        case["packed"] = "f32" if case["mode"] == "add" else rng.choice(("f32", "bf16"))
    return case


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _layout(specs):
    """One rank slice per tensor: (V, S, starts)."""
    S = max(-(-s.rows * s.cols // ALIGN) * ALIGN for s in specs)
    return len(specs), S, [i * S for i in range(len(specs))]


def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) * 7919 + 17)


def _grad_like(rows, cols, gen):
    """A gradient: a few strong directions over noise, 1e-3 in size."""
    r = max(1, min(16, rows // 4, cols // 4))
    low = torch.randn(rows, r, device=DEVICE, generator=gen) @ torch.randn(r, cols, device=DEVICE, generator=gen)
    return (low / math.sqrt(r) + torch.randn(rows, cols, device=DEVICE, generator=gen)) * 1e-3


def _distinct(n, rows):
    """How many different rows the tokens that _token_ids makes are expected to name."""
    r = torch.arange(rows, dtype=torch.float64)
    share = torch.log((r + 2) / (r + 1)) / math.log(rows)
    kept = n * 0.95 if n >= 20 else n
    return float((1 - torch.exp(kept * torch.log1p(-share.clamp(max=1 - 1e-12)))).sum())


def _token_ids(n, rows, idx, gen):
    """Token numbers by a power law over the table, a twentieth of them padding (-1) where there are many."""
    u = torch.rand(n, device=DEVICE, generator=gen, dtype=torch.float64)
    ids = ((rows ** u) - 1.0).floor().long().clamp_(0, rows - 1)
    ids = (ids * 7919 + 11) % rows          # common tokens are not the first rows
    if n >= 20:
        ids[torch.rand(n, device=DEVICE, generator=gen) < 0.05] = -1
    return ids if idx == "i64" else ids.int()


def prepare(case, seed):
    gen = _gen(seed)
    state = {"case": case}
    if case["op"] in ("ortho", "muon"):
        specs = [Spec(f"w{i}", r, c, "WHOLE") for i, (r, c) in enumerate(_shapes(case))]
    else:
        specs = [Spec("table", case["rows"], case["cols"], "ROWS", 1)]
    V, S, starts = _layout(specs)
    state.update(specs=specs, V=V, S=S, starts=starts)
    if own:
        import structure_aware_grouped_amd as rs
        state["plan"] = rs.rs_plan_load(specs, V, S, starts, device=torch.cuda.current_device())
    if case["op"] in ("ortho", "muon"):
        flat = torch.zeros(V * S, device=DEVICE)
        for s, at in zip(specs, starts):
            flat[at:at + s.rows * s.cols] = _grad_like(s.rows, s.cols, gen).reshape(-1)
        state["grad"] = flat.to(DTYPES[case["dt"]])
        del flat
        if case["op"] == "ortho":
            state["out"] = torch.zeros(V * S, dtype=torch.bfloat16, device=DEVICE)
        else:
            state["param"] = torch.randn(V * S, device=DEVICE, generator=gen) * 0.02
            state["momentum"] = torch.randn(V * S, device=DEVICE, generator=gen) * 2e-3
        if own:
            state["work"] = rs.rs_muon_workspace(state["plan"])
        return state
    n, cols, rows = case["tokens"], case["cols"], case["rows"]
    state["ids"] = _token_ids(n, rows, case["idx"], gen)
    if case["op"] == "embed":
        state["gathered"] = (torch.randn(V * S, device=DEVICE, generator=gen) * 0.02).to(DTYPES[case["dt"]])
        state["out"] = torch.zeros(n, cols, dtype=DTYPES[case["out"]], device=DEVICE)
        return state
    state["dy"] = (torch.randn(n, cols, device=DEVICE, generator=gen) * 1e-3).to(DTYPES[case["dt"]])
    if case["mode"] == "add":
        state["packed"] = torch.randn(V * S, device=DEVICE, generator=gen) * 1e-3
    else:
        state["packed"] = torch.zeros(V * S, dtype=DTYPES[case["packed"]], device=DEVICE)
    if own:
        state["work"] = rs.rs_embed_workspace(state["plan"], 0, n)
    return state


def _views(state, flat):
    return [flat[at:at + s.rows * s.cols].view(s.rows, s.cols) for s, at in zip(state["specs"], state["starts"])]


def _plain_orthogonal(g):
    """The Newton-Schulz iteration in 32 bits, on the matrix or its transpose, whichever is wide."""
    a, b, c = COEFFS
    x = g.T if g.shape[0] > g.shape[1] else g
    x = x * (1.0 / (g.double().square().sum().sqrt() + EPS)).float()
    for _ in range(STEPS):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if g.shape[0] > g.shape[1] else x


def _update_scale(rows, cols):
    """The root mean square of an AdamW update, 0.2, for an orthogonal rows x cols matrix."""
    return 0.2 * math.sqrt(max(rows, cols))


MOMENTUM = 0.95


def _plain(state):
    case = state["case"]
    if case["op"] == "ortho":
        for g, o in zip(_views(state, state["grad"]), _views(state, state["out"])):
            o.copy_(_plain_orthogonal(g.float()))
        return _views(state, state["out"])
    if case["op"] == "muon":
        for g, m, p in zip(*(_views(state, state[k]) for k in ("grad", "momentum", "param"))):
            g = g.float()
            m.mul_(MOMENTUM).add_(g)
            o = _plain_orthogonal(g + MOMENTUM * m if case["nesterov"] else m)
            p.mul_(1.0 - case["lr"] * case["wd"]).sub_(case["lr"] * _update_scale(*p.shape) * o)
        return {"param": _views(state, state["param"]), "momentum": _views(state, state["momentum"])}
    ids = state["ids"].long()
    named = (ids >= 0) & (ids < case["rows"])
    row = torch.where(named, ids, 0)
    if case["op"] == "embed":
        x = _views(state, state["gathered"])[0][row].float() * case["scale"]
        return torch.where(named[:, None], x, 0.0).to(DTYPES[case["out"]])
    dy = torch.where(named[:, None], state["dy"].float(), 0.0)
    total = torch.zeros(case["rows"], case["cols"], device=DEVICE).index_add_(0, row, dy)
    packed = _views(state, state["packed"])[0]
    if case["mode"] == "add":
        packed.add_(total * case["scale"])
    else:
        packed.copy_(total * case["scale"])
    return packed


def run(state):
    if not own:
        return _plain(state)
    import structure_aware_grouped_amd as rs
    case, plan = state["case"], state["plan"]
    if case["op"] == "ortho":
        rs.rs_orthogonalize(plan, state["grad"], state["out"], state["work"], coeffs=COEFFS, steps=STEPS, eps=EPS)
        return _views(state, state["out"])
    if case["op"] == "muon":
        rs.rs_muon_step(plan, state["param"], state["grad"], state["momentum"], state["work"], lr=case["lr"],
                        momentum_decay=MOMENTUM, weight_decay=case["wd"], nesterov=case["nesterov"], update_scale="rms",
                        coeffs=COEFFS, steps=STEPS, eps=EPS)
        return {"param": _views(state, state["param"]), "momentum": _views(state, state["momentum"])}
    if case["op"] == "embed":
        rs.rs_embed_rows(plan, 0, state["gathered"], state["ids"], state["out"], scale=case["scale"])
        return state["out"]
    rs.rs_embed_grad(plan, 0, state["ids"], state["dy"], state["packed"], state["work"],
                     prev=state["packed"] if case["mode"] == "add" else None, scale=case["scale"])
    return _views(state, state["packed"])[0]


def work(case):
    if case["op"] in ("ortho", "muon"):
        elems = sum(r * c for r, c in _shapes(case))
        # per step X X^T and A A^T are symmetric (half of each is computed), B X is whole
        flops = sum(STEPS * (3.0 * min(r, c) ** 2 * max(r, c) + min(r, c) ** 3) for r, c in _shapes(case))
        g = 4 if case["dt"] == "f32" else 2
        return {"bytes": elems * (g + 2.0 if case["op"] == "ortho" else g + 16.0), "flops": flops}
    n, cols, rows = case["tokens"], case["cols"], case["rows"]
    e = 4 if case["dt"] == "f32" else 2
    idx = 8 if case["idx"] == "i64" else 4
    if case["op"] == "embed":
        out = 4 if case["out"] == "f32" else 2
        # a row named twice is read once
        return {"bytes": n * idx + _distinct(n, rows) * cols * e + float(n) * cols * out, "flops": float(n) * cols}
    out = 4 if case["packed"] == "f32" else 2
    written = 2.0 * _distinct(n, rows) * cols * 4 if case["mode"] == "add" else float(rows) * cols * out
    return {"bytes": n * idx + float(n) * cols * e + written, "flops": float(n) * cols}


def exact(case, seed):
    """The outputs from the definitions, in 64 bits."""
    state = prepare(case, seed)

    def polynomial(g):
        # p(X X^T) X by Horner's rule, p(t) = a + t (b + c t)
        tall = g.shape[0] > g.shape[1]
        x = (g.mT if tall else g).contiguous()
        x = x / (torch.linalg.vector_norm(x) + EPS)
        eye = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
        a, b, c = COEFFS
        for _ in range(STEPS):
            gram = torch.mm(x, x.mT.contiguous())
            inner = torch.mm(gram, c * gram + b * eye) + a * eye
            x = torch.mm(inner, x)
        return x.mT if tall else x

    if case["op"] == "ortho":
        return [polynomial(g.double()) for g in _views(state, state["grad"])]
    if case["op"] == "muon":
        params, moms = [], []
        for g, m, p in zip(*(_views(state, state[k]) for k in ("grad", "momentum", "param"))):
            g, m, p = g.double(), m.double(), p.double()
            m = MOMENTUM * m + g
            o = polynomial(MOMENTUM * m + g if case["nesterov"] else m)
            params.append(p - case["lr"] * (case["wd"] * p + 0.2 * max(p.shape) ** 0.5 * o))
            moms.append(m)
        return {"param": params, "momentum": moms}
    ids = state["ids"].long()
    keep = torch.nonzero((ids >= 0) & (ids < case["rows"])).reshape(-1)
    if case["op"] == "embed":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=DEVICE)
        table = state["gathered"][:case["rows"] * case["cols"]].view(case["rows"], case["cols"])
        out[keep] = table.index_select(0, ids[keep]).double() * case["scale"]
        return out
    grad = torch.zeros(case["rows"], case["cols"], dtype=torch.float64, device=DEVICE)
    grad.index_add_(0, ids[keep], state["dy"][keep].double())
    grad *= case["scale"]
    if case["mode"] == "add":
        grad += state["packed"][:case["rows"] * case["cols"]].view(case["rows"], case["cols"]).double()
    return grad
