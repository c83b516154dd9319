"""The operators at the end of a model whose weights lie in a plan's flat buffers, as measurable cases.

Three operators, each with its gradient: layer norm (weight and bias read from
the gathered buffer, their gradients summed into the packed one), the softmax
cross entropy of a vocabulary head (the head's table read from the gathered
buffer, the logits never handed out, gradients of the inputs and of the table),
and distillation of that head from a teacher's top logits. Each case says how
large; ``run`` computes it in plain torch operations, or, where ``own`` is true,
by this package's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ALIGN = 16
EPS = 1e-5


class Spec:
    """One tensor of a group, with the fields the planner reads."""

    def __init__(self, name, rows, cols, kind, p0=0, p1=0):
        self.name, self.rows, self.cols, self.kind, self.p0, self.p1 = name, rows, cols, kind, p0, p1


def listed():
    return [
        # one token of a server's step: latency alone
        {"name": "norm 1 token", "op": "norm", "tokens": 1, "cols": 4096, "dt": "bf16", "out": "bf16", "center": False},
        # a training micro-batch of two 8192-token sequences
        {"name": "norm 16384 tokens", "op": "norm", "tokens": 16384, "cols": 8192, "dt": "bf16", "out": "bf16", "center": True},
        # the same micro-batch backwards, weight and bias gradients packed in fp32
        {"name": "norm grad 16384", "op": "norm_grad", "tokens": 16384, "cols": 8192, "dt": "bf16", "out": "bf16", "center": True, "packed": "f32", "prev": False},
        # an odd width with an fp32 residual stream, for a batch that is not full, added to earlier micro-batches
        {"name": "norm grad 4097 odd", "op": "norm_grad", "tokens": 4097, "cols": 1001, "dt": "f32", "out": "bf16", "center": True, "packed": "f32", "prev": True},
        # scoring a short continuation with a large vocabulary: reads the table once
        {"name": "loss 48 tokens", "op": "loss", "tokens": 48, "rows": 131072, "cols": 4096, "idx": "i64", "ignored": 0.0, "scale": 1.0},
        # evaluation of one 8192-token sequence
        {"name": "loss 8192 tokens", "op": "loss", "tokens": 8192, "rows": 131072, "cols": 4096, "idx": "i64", "ignored": 0.0, "scale": 1.0},
        # a small micro-batch, gradients packed for a bf16 reduce-scatter
        {"name": "loss grad 512", "op": "loss_grad", "tokens": 512, "rows": 32000, "cols": 4096, "idx": "i64", "ignored": 0.0, "scale": 1.0, "packed": "bf16", "prev": False},
        # fine-tuning on answers: half of the tokens belong to prompts and carry no loss; added to earlier micro-batches
        {"name": "loss grad 8192 answers", "op": "loss_grad", "tokens": 8192, "rows": 50000, "cols": 2880, "idx": "i32", "ignored": 0.5, "scale": 1.0, "packed": "f32", "prev": True},
        # the training micro-batch of two 8192-token sequences with the largest table
        {"name": "loss grad 16384", "op": "loss_grad", "tokens": 16384, "rows": 131072, "cols": 4096, "idx": "i64", "ignored": 0.0, "scale": 1.0, "packed": "f32", "prev": False},
        # how far a student is from its teacher, on a validation batch
        {"name": "distill 2048 top 64", "op": "distill", "tokens": 2048, "rows": 32000, "cols": 4096, "idx": "i32", "top": 64, "teacher": "bf16", "temperature": 1.0},
        # a distillation micro-batch at a raised temperature
        {"name": "distill grad 4096 top 64", "op": "distill_grad", "tokens": 4096, "rows": 131072, "cols": 4096, "idx": "i32", "top": 64, "teacher": "bf16", "temperature": 2.0, "packed": "f32", "prev": False},
        # an odd table and batch, few teacher logits
        {"name": "distill grad 517 odd", "op": "distill_grad", "tokens": 517, "rows": 32001, "cols": 1001, "idx": "i64", "top": 7, "teacher": "f32", "temperature": 1.0, "packed": "bf16", "prev": True},
    ]


def _log(rng, lo, hi):
    """A whole number spread over its logarithm, ends included, odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "loss", "loss_grad", "distill", "distill_grad"))
    packed = {"packed": rng.choice(("f32", "bf16")), "prev": rng.random() < 0.4}
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            cols = max(64, cols // 64 * 64)
        case = {"op": op, "tokens": min(_log(rng, 1, 65536), (1 << 27) // cols), "cols": cols, "dt": rng.choice(("f32", "bf16")),
                "out": rng.choice(("f32", "bf16")), "center": rng.random() < 0.5}
        if op == "norm_grad":
            case.update(packed)
        return case
    rows, cols = _log(rng, 1000, 131072), _log(rng, 64, 8192)
    if rng.random() < 0.6:
        cols = max(64, cols // 64 * 64)
    if rng.random() < 0.4:
        rows = max(1024, rows // 64 * 64)
    rows = min(rows, (1 << 29) // cols)
    case = {"op": op, "tokens": min(_log(rng, 1, 16384), (1 << 43) // (rows * cols)), "rows": rows, "cols": cols, "idx": rng.choice(("i64", "i32"))}
    if op.startswith("loss"):
        case.update(ignored=rng.choice((0.0, round(rng.uniform(0.05, 0.9), 2))), scale=rng.choice((1.0, round(rng.uniform(0.5, 1.5), 3))))
    else:
        case.update(top=_log(rng, 1, 100), teacher=rng.choice(("f32", "bf16")), temperature=rng.choice((1.0, 2.0, round(rng.uniform(0.7, 4.0), 2))))
    if op.endswith("grad"):
        case.update(packed)
    return case


def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) * 7919 + 17)


def _specs(case):
    if case["op"].startswith("norm"):
        return [Spec("weight", case["cols"], 1, "ROWS", 1)] + ([Spec("bias", case["cols"], 1, "ROWS", 1)] if case["center"] else [])
    return [Spec("head", case["rows"], case["cols"], "ROWS", 1)]


def _layout(specs):
    """One rank slice per tensor: (V, S, starts)."""
    S = max(-(-s.rows * s.cols // ALIGN) * ALIGN for s in specs)
    return len(specs), S, [i * S for i in range(len(specs))]


def _views(state, flat):
    return [flat[at:at + s.rows * s.cols].view(s.rows, s.cols) for s, at in zip(state["specs"], state["starts"])]


def _prepare_packed(state, gen):
    case, n = state["case"], state["V"] * state["S"]
    state["packed"] = torch.zeros(n, dtype=DTYPES[case["packed"]], device=DEVICE)
    state["prev"] = torch.randn(n, device=DEVICE, generator=gen) * 1e-3 if case["prev"] else None


def prepare(case, seed):
    gen = _gen(seed)
    specs = _specs(case)
    V, S, starts = _layout(specs)
    state = {"case": case, "specs": specs, "V": V, "S": S, "starts": starts}
    if own:
        import structure_aware_grouped_amd as rs
        state["plan"] = rs.rs_plan_load(specs, V, S, starts, device=torch.cuda.current_device())
    n, cols, grad = case["tokens"], case["cols"], case["op"].endswith("grad")
    randn = lambda *shape: torch.randn(*shape, device=DEVICE, generator=gen)  # noqa: E731
    if case["op"].startswith("norm"):
        gathered = torch.zeros(V * S, device=DEVICE)
        gathered[:cols] = 1.0 + 0.2 * randn(cols)
        if case["center"]:
            gathered[S:S + cols] = 0.1 * randn(cols)
        state["gathered"] = gathered.to(torch.bfloat16)
        # a residual stream: tokens of different sizes, a mean, and a few columns far above the others
        x = randn(n, cols) * torch.exp(0.5 * randn(n, 1)) + 0.3 * randn(n, 1)
        x[:, :: max(1, cols // 8)] *= 8.0
        state["x"] = x.to(DTYPES[case["dt"]])
        state["y"] = torch.zeros(n, cols, dtype=DTYPES[case["out"]], device=DEVICE)
        if grad:
            state["dy"] = (randn(n, cols) * 1e-3).to(DTYPES[case["out"]])
            state["dx"] = torch.zeros(n, cols, dtype=DTYPES[case["dt"]], device=DEVICE)
            _prepare_packed(state, gen)
            if own:
                state["work"] = rs.rs_layer_norm_workspace(state["plan"], 0, n)
        return state
    rows = case["rows"]
    state["gathered"] = (randn(V * S) * (1.28 / math.sqrt(cols))).to(torch.bfloat16)
    table = _views(state, state["gathered"])[0]
    named = torch.randint(0, rows, (n,), device=DEVICE, generator=gen)
    # normed hidden states that lean towards one row of the table, from not at all to almost surely
    lean = torch.rand(n, 1, device=DEVICE, generator=gen) * (math.log(rows) + 4.0) / 1.64
    state["x"] = (randn(n, cols) + lean * table[named].float()).to(torch.bfloat16)
    idx = torch.int64 if case["idx"] == "i64" else torch.int32
    if case["op"].startswith("loss"):
        other = torch.randint(0, rows, (n,), device=DEVICE, generator=gen)
        targets = torch.where(torch.rand(n, device=DEVICE, generator=gen) < 0.7, named, other)
        if case["ignored"]:
            targets[torch.rand(n, device=DEVICE, generator=gen) < case["ignored"]] = -100
        state["targets"] = targets.to(idx)
    else:
        k = min(case["top"], rows)
        step = torch.randint(1, rows // k + 1, (n, 1), device=DEVICE, generator=gen)
        ids = (named[:, None] + step * torch.arange(k, device=DEVICE)) % rows
        logits = 12.0 - 2.0 * torch.log1p(torch.arange(k, device=DEVICE, dtype=torch.float32)) + 0.5 * randn(n, k)
        # a teacher that kept fewer logits for some tokens leaves the places behind them empty
        kept = torch.randint(1, k + 1, (n, 1), device=DEVICE, generator=gen)
        kept[torch.rand(n, 1, device=DEVICE, generator=gen) < 0.8] = k
        state["ids"] = torch.where(torch.arange(k, device=DEVICE) < kept, ids, -1).to(idx).contiguous()
        state["logits"] = logits.to(DTYPES[case["teacher"]])
    state["loss"] = torch.zeros(n, device=DEVICE)
    if grad:
        # each token's share of the batch's mean, longer answers weighing less per token
        state["weights"] = (0.5 + torch.rand(n, device=DEVICE, generator=gen)) / n
        state["dx"] = torch.zeros(n, cols, dtype=torch.bfloat16, device=DEVICE)
        _prepare_packed(state, gen)
    if own:
        state["work"] = rs.rs_head_workspace(state["plan"], 0, n, top=case.get("top", 0), packed=state.get("packed"))
    return state


def _plain_pack(state, grads):
    """[prev +] the gradients, rounded to the packed buffer's type."""
    out = _views(state, state["packed"])
    before = _views(state, state["prev"]) if state["prev"] is not None else [None] * len(out)
    for o, p, g in zip(out, before, grads):
        o.copy_((g if p is None else p + g.view_as(p)).view_as(o))
    return out


def _plain_norm(state):
    case = state["case"]
    params = [p.reshape(-1).float() for p in _views(state, state["gathered"])]
    x = state["x"].float()
    if case["center"]:
        x = x - x.mean(1, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    hat = x * r
    if case["op"] == "norm":
        y = hat * params[0]
        state["y"].copy_(y + params[1] if case["center"] else y)
        return state["y"]
    dy = state["dy"].float()
    g = dy * params[0]
    dx = g - hat * (g * hat).mean(1, keepdim=True)
    if case["center"]:
        dx = dx - g.mean(1, keepdim=True)
    state["dx"].copy_(dx * r)
    return {"dx": state["dx"], "packed": _plain_pack(state, [(dy * hat).sum(0), dy.sum(0)][:len(params)])}


def _plain_head(state):
    case, grad = state["case"], state["case"]["op"].endswith("grad")
    n, rows = case["tokens"], case["rows"]
    table, x = _views(state, state["gathered"])[0].float(), state["x"].float()
    if case["op"].startswith("loss"):
        t, scale, factor = 1.0, case["scale"], 1.0
        ids = state["targets"].long()[:, None]
        given = (ids >= 0) & (ids < rows)
        q = given.float()
    else:
        t, scale, factor = case["temperature"], 1.0, case["temperature"] ** 2
        ids = state["ids"].long()
        given = (ids >= 0) & (ids < rows)
        z = torch.where(given, state["logits"].float() / t, -math.inf)
        q = torch.exp(z - z.max(1, keepdim=True).values)
        q = torch.nan_to_num(q / q.sum(1, keepdim=True), nan=0.0)
    some = given.any(1)
    logits = (x @ table.T) * (scale / t)
    top = logits.max(1, keepdim=True).values
    p = torch.exp(logits - top)
    total = p.sum(1, keepdim=True)
    at = torch.where(given, ids, 0)
    log_p = logits.gather(1, at) - top - torch.log(total)
    loss = factor * torch.where(given & (q > 0), q * (torch.log(torch.where(q > 0, q, 1.0)) - log_p), 0.0).sum(1)
    state["loss"].copy_(torch.where(some, loss, 0.0))
    if not grad:
        return state["loss"]
    del logits
    p /= total
    p.scatter_add_(1, at, torch.where(given, -q, 0.0))
    p *= torch.where(some, state["weights"] * (factor * scale / t), 0.0)[:, None]
    state["dx"].copy_(p @ table)
    return {"loss": state["loss"], "dx": state["dx"], "packed": _plain_pack(state, [p.T @ x])}


def run(state):
    case = state["case"]
    if not own:
        return _plain_norm(state) if case["op"].startswith("norm") else _plain_head(state)
    import structure_aware_grouped_amd as rs
    plan = state["plan"]
    if case["op"] == "norm":
        rs.rs_layer_norm(plan, 0, state["gathered"], state["x"], state["y"], bias=1 if case["center"] else None, eps=EPS,
                         center=case["center"])
        return state["y"]
    if case["op"] == "norm_grad":
        rs.rs_layer_norm_grad(plan, 0, state["gathered"], state["x"], state["dy"], state["dx"], state["packed"], state["work"],
                              bias=1 if case["center"] else None, eps=EPS, center=case["center"], prev=state["prev"])
        return {"dx": state["dx"], "packed": _views(state, state["packed"])}
    if case["op"] == "loss":
        rs.rs_head_loss(plan, 0, state["gathered"], state["x"], state["targets"], state["loss"], state["work"], scale=case["scale"])
        return state["loss"]
    if case["op"] == "distill":
        rs.rs_distill_loss(plan, 0, state["gathered"], state["x"], state["ids"], state["logits"], state["loss"], state["work"],
                           temperature=case["temperature"])
        return state["loss"]
    if case["op"] == "loss_grad":
        rs.rs_head_grad(plan, 0, state["gathered"], state["x"], state["targets"], state["loss"], state["dx"], state["packed"],
                        state["work"], weights=state["weights"], prev=state["prev"], scale=case["scale"])
    else:
        rs.rs_distill_grad(plan, 0, state["gathered"], state["x"], state["ids"], state["logits"], state["loss"], state["dx"],
                           state["packed"], state["work"], weights=state["weights"], prev=state["prev"],
                           temperature=case["temperature"])
    return {"loss": state["loss"], "dx": state["dx"], "packed": _views(state, state["packed"])}


def work(case):
    n, cols, grad = float(case["tokens"]), float(case["cols"]), case["op"].endswith("grad")
    size = {"f32": 4.0, "bf16": 2.0}
    if case["op"].startswith("norm"):
        e, o, params = size[case["dt"]], size[case["out"]], 2 if case["center"] else 1
        if not grad:
            return {"bytes": n * cols * (e + o) + params * cols * 2, "flops": 8 * n * cols}
        packed = params * cols * (size[case["packed"]] + (4.0 if case["prev"] else 0.0))
        return {"bytes": n * cols * (2 * e + o) + cols * 2 + packed, "flops": 16 * n * cols}
    rows = float(case["rows"])
    # a token without a target takes part in no product
    kept = n * (1.0 - case.get("ignored", 0.0))
    small = n * (4.0 + (8.0 if case["idx"] == "i64" else 4.0) * case.get("top", 1))
    if case["op"].startswith("distill"):
        small += n * case["top"] * size[case["teacher"]]
    if not grad:
        return {"bytes": rows * cols * 2 + kept * cols * 2 + small, "flops": 2 * kept * rows * cols}
    packed = rows * cols * (size[case["packed"]] + (4.0 if case["prev"] else 0.0))
    return {"bytes": rows * cols * 2 + kept * cols * 2 + n * (cols * 2 + 4) + small + packed, "flops": 6 * kept * rows * cols}


def _exact_pack(state, grads):
    prev = _views(state, state["prev"]) if state["prev"] is not None else None
    return [(g.reshape(s.rows, s.cols) + (prev[i].double() if prev else 0.0)) for i, (g, s) in enumerate(zip(grads, state["specs"]))]


def exact(case, seed):
    """The outputs from the definitions, in 64 bits, some tokens at a time."""
    state = prepare(case, seed)
    n, cols, grad = case["tokens"], case["cols"], case["op"].endswith("grad")
    f64 = dict(dtype=torch.float64, device=DEVICE)
    params = [p.double() for p in _views(state, state["gathered"])]
    if case["op"].startswith("norm"):
        w = params[0].reshape(-1)
        block = max(1, (1 << 26) // cols)
        out, dw, db = torch.empty(n, cols, **f64), torch.zeros(cols, **f64), torch.zeros(cols, **f64)
        for i in range(0, n, block):
            x = state["x"][i:i + block].double()
            mean = x.sum(1, keepdim=True) / cols if case["center"] else 0.0
            dev = ((x - mean).square().sum(1, keepdim=True) / cols + EPS).sqrt()
            hat = (x - mean) / dev
            if not grad:
                out[i:i + block] = hat * w + (params[1].reshape(-1) if case["center"] else 0.0)
                continue
            dy = state["dy"][i:i + block].double()
            dw += (dy * hat).sum(0)
            db += dy.sum(0)
            # the Jacobian of the norm: the identity less the projections on hat (and on ones), over the deviation
            g = dy * w
            along = (g * hat).sum(1, keepdim=True) / cols
            out[i:i + block] = (g - along * hat - (g.sum(1, keepdim=True) / cols if case["center"] else 0.0)) / dev
        return {"dx": out, "packed": _exact_pack(state, [dw, db][:len(params)])} if grad else out
    table, rows = params[0], case["rows"]
    loss = torch.zeros(n, **f64)
    dx = torch.zeros(n, cols, **f64)
    dtable = torch.zeros(rows, cols, **f64) if grad else None
    block = max(1, (1 << 28) // rows)
    for i in range(0, n, block):
        x = state["x"][i:i + block].double()
        if "targets" in state:
            ids, t, scale = state["targets"][i:i + block].long()[:, None], 1.0, case["scale"]
            there = (ids >= 0) & (ids < rows)
            q = there.double()
        else:
            ids, t, scale = state["ids"][i:i + block].long(), case["temperature"], 1.0
            there = (ids >= 0) & (ids < rows)
            q = torch.softmax((state["logits"][i:i + block].double() / t).masked_fill(~there, -math.inf), 1).nan_to_num(0.0)
        full = torch.zeros(x.shape[0], rows, **f64).scatter_add_(1, ids.clamp(0, rows - 1), q * there)
        live = there.any(1).double()
        s = torch.mm(x, table.mT.contiguous()) * (scale / t)
        log_p = s - torch.logsumexp(s, 1, keepdim=True)
        del s
        # the teacher's entropy comes from its own places, for a row named twice counts as its sum
        h = torch.special.xlogy(q, q).sum(1)
        loss[i:i + block] = t * t * live * (h - (full * log_p).sum(1))
        if grad:
            d = (log_p.exp() - full) * (live * state["weights"][i:i + block].double() * (t * scale))[:, None]
            del log_p, full
            dx[i:i + block] = torch.mm(d, table)
            dtable += torch.mm(d.mT.contiguous(), x)
    return {"loss": loss, "dx": dx, "packed": _exact_pack(state, [dtable])} if grad else loss
