"""Losses and gradients of tokens that the head is sure of: logits of 25 to 200,
with nearly all of the softmax on the target.

x of token t is the unit vector of column t, so its logits are the table's
column t: exact, and only what is done with them can be off. Tolerances, with
u = 2^-24 (half an fp32 step). Of 700 or 5000 logits a token has four that
count (its target's and three others, 8 to 20 below), the rest underflow. The
sum of their exponentials, near 1, is off by 4 u (an exponential), by u for each
of four additions and for each of four partial sums joined: 12 u, and so is its
logarithm. A difference of a logit and the largest is exact but for u of itself,
which the exponential of that difference damps. -log p of the target is then off
by 16 u at most, whatever the logits' size, and is never negative; a target that
lies `gap` below by 16 u (1 + gap). p of the target is off by 24 u; of another
row by 24 u and 2 u per unit of its gap, of itself; p - q is rounded to 22 bits
or to within 2^-38 of the largest weight."""
import numpy as np
import pytest
import torch

from oracle import head as OH
from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def _inputs(rs, n, rows, cols, largest, seed=0):
    rng = np.random.default_rng(seed + n)
    specs = [TensorSpec("head", rows, cols, "ROWS", 1)]
    S, starts, _, _ = rs.rs_plan_build(specs, 2)
    plan = rs.rs_plan_load(specs, 2, S, starts, 2, 0)
    table = np.full((rows, cols), -200.0)
    named = np.empty((n, 4), dtype=np.int64)
    gap = np.zeros((n, 4))
    for t in range(n):
        named[t] = rng.choice(rows, 4, replace=False)
        gap[t, 1:] = rng.integers(8, 21, 3)
        table[named[t], t] = largest - gap[t]
    flat = torch.zeros(2 * S, dtype=torch.bfloat16)
    at = slice(starts[0], starts[0] + rows * cols)
    flat[at] = torch.from_numpy(table.ravel()).to(torch.bfloat16)
    assert np.array_equal(flat[at].double().numpy().reshape(rows, cols), table)      # multiples of bf16's steps
    x = torch.zeros(n, cols, dtype=torch.bfloat16)
    x[torch.arange(n), torch.arange(n)] = 1.0
    weights = torch.from_numpy(0.5 + 0.5 * rng.random(n)).float()
    return plan, at, flat.to(DEV), x.to(DEV), table, named, gap, weights.to(DEV), rng


SIZES = [(64, 700, 64), (120, 5000, 128), (300, 700, 320)]


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("largest", [25.0, 50.0, 100.0, 200.0])
@pytest.mark.parametrize("top", [0, 1, 3])
def test_loss(gpu_lib, n, rows, cols, largest, top):
    import structure_aware_grouped_amd as rs
    plan, _, flat, x, table, named, gap, _, rng = _inputs(rs, n, rows, cols, largest)
    loss, temperature = torch.full((n,), float("nan"), device=DEV), 1.0
    work = rs.rs_head_workspace(plan, 0, n, top=top)
    if top:
        ids, temperature = named[:, :top].copy(), 2.0
        teacher = torch.from_numpy(rng.standard_normal((n, top)) - 4.0 * np.arange(top)).float().to(DEV)
        rs.rs_distill_loss(plan, 0, flat, x, torch.from_numpy(ids).to(DEV), teacher, loss, work, temperature=temperature, scale=2.0)
        want, _, full, _ = OH.losses(x.double().cpu().numpy(), table, ids, teacher.double().cpu().numpy(), temperature, 2.0)
        q, _ = OH.shares(ids, rows, teacher.double().cpu().numpy(), temperature)
        # q by 8 u and 16 u per unit of the logits' spread (under 16), which its logarithm and the gap multiply
        off = temperature ** 2 * U * (16 + (q * 16 * (1 + gap[:, :top])).sum(1) + (q * 264 * (gap[:, :top] + 1 - np.log(q))).sum(1) * (top > 1))
    else:
        rs.rs_head_loss(plan, 0, flat, x, torch.from_numpy(named[:, 0].copy()).to(DEV), loss, work)
        want = OH.losses(x.double().cpu().numpy(), table, named[:, :1])[0]
        off = 16 * U
    got = loss.double().cpu().numpy()
    assert (np.abs(got - want) <= off).all(), np.abs(got - want).max() / U
    if top < 2:
        assert (got >= 0).all()
    plan.close()


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("largest", [25.0, 100.0, 200.0])
@pytest.mark.parametrize("top", [0, 1])
def test_gradients(gpu_lib, n, rows, cols, largest, top):
    """The table's gradient in column t is that of token t's logits; the loss is that of the call without gradients."""
    import structure_aware_grouped_amd as rs
    plan, at, flat, x, table, named, gap, weights, _ = _inputs(rs, n, rows, cols, largest)
    ids = torch.from_numpy(named[:, :1].copy()).to(DEV)
    loss, alone, dx = torch.empty(n, device=DEV), torch.empty(n, device=DEV), torch.empty_like(x)
    packed = torch.full((2 * plan.S,), float("nan"), device=DEV)
    work = rs.rs_head_workspace(plan, 0, n, top=top, packed=packed)
    if top:
        teacher = torch.zeros(n, 1, device=DEV)
        rs.rs_distill_grad(plan, 0, flat, x, ids, teacher, loss, dx, packed, work, weights=weights)
        rs.rs_distill_loss(plan, 0, flat, x, ids, teacher, alone, work)
    else:
        rs.rs_head_grad(plan, 0, flat, x, ids[:, 0].contiguous(), loss, dx, packed, work, weights=weights)
        rs.rs_head_loss(plan, 0, flat, x, ids[:, 0].contiguous(), alone, work)
    assert torch.equal(loss, alone) and bool((loss >= 0).all())
    _, p, full, _ = OH.losses(x.double().cpu().numpy(), table, named[:, :1])
    w = weights.double().cpu().numpy()
    want = (w[:, None] * (p - full)).T
    distance = np.full((n, rows), 0.0)
    distance[np.arange(n)[:, None], named] = gap
    off = w[:, None] * (24 * U * (full + p) + 2 * U * distance * p + 2.0 ** -22 * np.abs(p - full)) + w.max() * 2.0 ** -38
    got = packed[at].double().cpu().numpy().reshape(rows, cols)[:, :n]
    bad = np.abs(got - want) > off.T
    assert not bad.any(), (bad.sum(), (np.abs(got - want) / U).max())
    plan.close()
