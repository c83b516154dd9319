"""The operators of a model's two ends together, as a training step calls them:
rows of a tied table (rs_embed_rows), layer norm, the head's loss and gradients,
layer norm's gradients, and the rows' gradient added onto the head's in the
packed buffer.

Tolerances. The looked-up rows are exact, so x, r and h of layer norm are. Three
roundings to bf16 (2^-8) lie on the way: y, the head's dx, layer norm's dx. The
bounds follow each through absolute values: y through the logits (c sum |W| |y|
2^-8) into p (p times that and its mean) and the table's gradient; the head's dx
through layer norm's gradient (|dx| off by r (|g| + mean |g| + |h| mean |h g|)
of the g that is off); all of them added up over the tokens of a row. The head's
own rounding of p - q is one of 2^-8 for dx and one of 2^-22 for the table. fp32
sums of at most 600 values add 600 * 2^-23 = 2^-13.8 of the sums of absolute
values, products of bounds (second order) at most 2^-8 * (1 + 6) of the bounds:
together under 2^-4 of the bounds and 2^-13 of the sums."""
import os
import re
import textwrap

import numpy as np
import pytest
import torch

from oracle import head as OH, norm as ON
from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STEP = 2.0 ** -8
ROWS, COLS, V = 600, 136, 3


class Model:
    """A tied table, a layer norm and the buffers of one step."""

    def __init__(self, rs, n, top, seed=0):
        rng = np.random.default_rng(seed)
        specs = [TensorSpec("table", ROWS, COLS, "ROWS", 1), TensorSpec("w", COLS, 1, "ROWS", 1), TensorSpec("b", 1, COLS, "WHOLE")]
        S, self.starts, _, _ = rs.rs_plan_build(specs, V)
        self.plan = rs.rs_plan_load(specs, V, S, self.starts, V, 0)
        self.numels = [ROWS * COLS, COLS, COLS]
        flat = torch.zeros(V * S)
        for t, (mean, dev) in enumerate(((0.0, 1.0), (1.0, 0.3), (0.0, 0.3))):
            flat[self.part(t)] = torch.from_numpy(mean + dev * rng.standard_normal(self.numels[t])).float()
        self.gathered = flat.to(DEV, torch.bfloat16)
        ids = rng.integers(0, ROWS, n)
        ids[: n // 3] = ids[0]                          # one row many times
        ids[rng.random(n) < 0.1] = -1                   # padding: no row, no target
        self.ids = torch.from_numpy(ids).to(DEV)
        target = rng.integers(0, ROWS, (n, max(top, 1)))
        target[ids < 0] = -100
        self.target = torch.from_numpy(target if top else target[:, 0].copy()).to(DEV)
        self.teacher = torch.from_numpy(rng.standard_normal((n, top)) * 2).to(DEV, torch.bfloat16) if top else None
        self.weights = torch.from_numpy((ids >= 0) / max((ids >= 0).sum(), 1)).float().to(DEV)
        self.n, self.top, self.scale, self.temperature = n, top, 0.25, 2.0 if top else 1.0
        b = dict(dtype=torch.bfloat16, device=DEV)
        self.x, self.y, self.dy, self.dx = (torch.empty(n, COLS, **b) for _ in range(4))
        self.loss = torch.empty(n, device=DEV)
        self.packed = torch.full((V * S,), 7.0, device=DEV)
        self.head_work = rs.rs_head_workspace(self.plan, 0, n, top=top, packed=self.packed)
        self.norm_work = rs.rs_layer_norm_workspace(self.plan, 1, n)
        self.row_work = rs.rs_embed_workspace(self.plan, 0, n)

    def part(self, t):
        return slice(self.starts[t], self.starts[t] + self.numels[t])

    def step(self, rs):
        p, g = self.plan, self.gathered
        rs.rs_embed_rows(p, 0, g, self.ids, self.x)
        rs.rs_layer_norm(p, 1, g, self.x, self.y, bias=2)
        if self.top:
            rs.rs_distill_grad(p, 0, g, self.y, self.target, self.teacher, self.loss, self.dy, self.packed, self.head_work,
                               temperature=self.temperature, scale=self.scale, weights=self.weights, inv_v=True)
        else:
            rs.rs_head_grad(p, 0, g, self.y, self.target, self.loss, self.dy, self.packed, self.head_work, scale=self.scale,
                            weights=self.weights, inv_v=True)
        rs.rs_layer_norm_grad(p, 1, g, self.x, self.dy, self.dx, self.packed, self.norm_work, bias=2, inv_v=True)
        rs.rs_embed_grad(p, 0, self.ids, self.dx, self.packed, self.row_work, prev=self.packed, inv_v=True)

    def expect(self):
        """The packed gradients of the three tensors in 64 bits, their bounds, loss and its bound."""
        f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        table, w, b = (f64(self.gathered[self.part(t)]) for t in range(3))
        table, ids, target, weight = table.reshape(ROWS, COLS), f64(self.ids).astype(int), self.target.cpu().numpy(), f64(self.weights)
        teacher = None if self.teacher is None else f64(self.teacher)
        x = np.where(ids[:, None] >= 0, table[np.maximum(ids, 0)], 0.0)
        h, r = ON._parts(x, 1e-5, True)
        y = h * w + b
        loss, p, q, live = OH.losses(y, table, target, teacher, self.temperature, self.scale)
        dy, dtable, _, _ = OH.gradients(y, table, target, weight, teacher, self.temperature, self.scale)
        dx, dw, db = ON.norm_grad(x, dy, w, 1e-5, True)
        off_y = STEP * np.abs(y)
        off_l = self.scale / self.temperature * off_y @ np.abs(table).T
        off_loss = self.temperature ** 2 * ((p + q) * off_l).sum(1) * live
        a = np.abs(weight * self.scale * self.temperature)[:, None] * live[:, None]
        off_d = a * p * (off_l + (p * off_l).sum(1, keepdims=True))
        d = a * np.abs(p - q)
        off_dy = (off_d + STEP * d) @ np.abs(table) + STEP * np.abs(dy)
        off_g = off_dy * np.abs(w)
        off_dx = r * (off_g + off_g.mean(1, keepdims=True) + np.abs(h) * (np.abs(h) * off_g).mean(1, keepdims=True)) + STEP * np.abs(dx)
        named = ids >= 0
        sums, off = np.zeros_like(table), np.zeros_like(table)
        np.add.at(sums, ids[named], dx[named])
        np.add.at(off, ids[named], off_dx[named])
        off += off_d.T @ np.abs(y) + (d + off_d).T @ off_y
        whole = d.T @ np.abs(y)
        np.add.at(whole, ids[named], np.abs(dx[named]))
        sigma = float(np.float32(1.0) / np.float32(V))
        return ([sigma * v for v in (dtable + sums, dw, db)],
                [sigma * (1.0625 * o + 2.0 ** -13 * s)
                 for o, s in ((off, whole), ((np.abs(h) * off_dy).sum(0), (np.abs(h) * np.abs(dy)).sum(0)), (off_dy.sum(0), np.abs(dy).sum(0)))],
                loss, 1.0625 * off_loss + 2.0 ** -13 * (np.abs(loss) + np.log(ROWS)))


@pytest.mark.parametrize("n,top", [(1, 0), (40, 0), (300, 0), (40, 12), (300, 12)])
def test_a_step_of_both_ends(gpu_lib, n, top):
    import structure_aware_grouped_amd as rs
    m = Model(rs, n, top)
    m.step(rs)
    torch.cuda.synchronize()
    want, off, loss, off_loss = m.expect()
    assert (np.abs(m.loss.double().cpu().numpy() - loss) <= off_loss).all()
    got = m.packed.double().cpu().numpy()
    for t in range(3):
        assert (np.abs(got[m.part(t)] - want[t].ravel()) <= off[t].ravel() + 2.0 ** -40).all(), t
    left = np.ones(got.size, dtype=bool)
    for t in range(3):
        left[m.part(t)] = False
    assert (got[left] == 7.0).all()
    first = m.packed.clone()
    m.packed.fill_(-3.0)
    m.step(rs)
    for t in range(3):
        assert torch.equal(m.packed[m.part(t)], first[m.part(t)])
    m.plan.close()


@pytest.mark.parametrize("top", [0, 5])
def test_a_step_in_a_graph(gpu_lib, top):
    """Captured once and replayed on new inputs, with eager steps of the same buffers between the replays."""
    import structure_aware_grouped_amd as rs
    m, ref = Model(rs, 200, top), Model(rs, 200, top)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        m.step(rs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step(rs)
    for i in range(4):
        other = Model(rs, 200, top, seed=10 + i)
        for own in (m, ref):
            for name in ("gathered", "ids", "target", "weights") + (("teacher",) if top else ()):
                getattr(own, name).copy_(getattr(other, name))
        other.plan.close()
        torch.cuda.synchronize()
        graph.replay()
        ref.step(rs)
        torch.cuda.synchronize()
        assert torch.equal(m.packed, ref.packed) and torch.equal(m.loss, ref.loss)
        m.step(rs)
        torch.cuda.synchronize()
        assert torch.equal(m.packed, ref.packed)
    del graph
    m.plan.close()
    ref.plan.close()


def test_the_readme_example_of_these_calls_runs(gpu_lib):
    """And its losses and the table's gradient hold against torch's operations in fp32."""
    import structure_aware_grouped_amd as rs
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    block = re.search(r"tied to the lookup's \(imports as above\):\n\n((?:    .*\n|\n)+)", text).group(1)
    env = {"torch": torch, "rs": rs, "TensorSpec": TensorSpec}
    exec(compile(textwrap.dedent(block), "README.md", "exec"), env)
    torch.cuda.synchronize()
    start = env["starts"][0]
    table = env["gathered"][start:start + 32000 * 4096].view(32000, 4096).double()
    y, target, at = env["y"].double(), env["targets"], torch.arange(64, device=DEV)
    got = env["packed"][start:start + 32000 * 4096].view(32000, 4096)
    total = torch.zeros(32000, 4096, device=DEV, dtype=torch.float64)
    for t0 in range(0, 2048, 64):
        l = 2.0 ** -6 * y[t0:t0 + 64] @ table.T
        # 4096 products of normal values: sums of absolute values of 2^-6 * 4096 * 2 / pi = 41, under 60; 2 * 4098 u of
        # them is 0.03. Partial sums stay under 10 (deviation 1): 256 additions of two half steps of those are 3.1e-4
        want = l.logsumexp(1) - l[at, target[t0:t0 + 64]]
        assert float((env["loss"][t0:t0 + 64].double() - want).abs().max()) <= 2 * 3.1e-4 + 200 * 2.0 ** -24
        d = l.softmax(1)
        d[at, target[t0:t0 + 64]] -= 1.0
        total += 2.0 ** -6 * d.T @ y[t0:t0 + 64]
    # d is off by at most 2 * 3.1e-4 of p, so the gradient by that of the sums: in the Frobenius norm under 2^-9 of it
    assert float((got.double() - total).norm() / total.norm()) <= 2.0 ** -9
