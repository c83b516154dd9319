"""dx where a token's targets are most of p - q: what its rounding to bf16 leaves
there is added in fp32, so dx is within half a step of its own bf16 of the exact
one.

Only four rows of the table hold anything, and they are the targets; x is small,
so the softmax is nearly flat. Tolerances, with u = 2^-24: p is off by 100 u of
itself and so is q; p of the rows that are no target of the token is rounded to
bf16 (2^-8 of it, at most three rows of 300); the fp32 sums have at most eight
terms that are not 0 (16 u of their absolute values). The result is rounded once,
by half of the step at its size. With a p - q rounded to bf16 at the targets too,
the results would be off by more in a part of the elements, which the test shows
in 64 bits on the host."""
import numpy as np
import pytest
import torch

from oracle import head as OH
from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
ROWS, HELD = 300, np.array([0, 77, 150, 299])


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).double().numpy()


def _half_step(a):
    """Half of bf16's step at |a|: 2^-8 of the power of two below."""
    return np.where(a == 0, 0.0, 2.0 ** (np.floor(np.log2(np.where(a == 0, 1.0, np.abs(a)))) - 8))


@pytest.mark.parametrize("packed_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,cols", [(1, 256), (40, 72), (100, 320), (300, 256)])
@pytest.mark.parametrize("kind", ["labels", "teacher", "teacher twice"])
def test_dx_is_within_its_own_rounding(gpu_lib, packed_dt, n, cols, kind):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(n + cols)
    specs = [TensorSpec("head", ROWS, cols, "ROWS", 1)]
    S, starts, _, _ = rs.rs_plan_build(specs, 2)
    plan = rs.rs_plan_load(specs, 2, S, starts, 2, 0)
    table = np.zeros((ROWS, cols))
    table[HELD] = _bf16(rng.standard_normal((4, cols)))
    flat = torch.zeros(2 * S)
    flat[starts[0]:starts[0] + ROWS * cols] = torch.from_numpy(table.ravel())
    flat = flat.to(DEV, torch.bfloat16)
    x = torch.from_numpy(rng.standard_normal((n, cols)) * 2.0 ** -7).to(DEV, torch.bfloat16)
    weights = torch.from_numpy(0.5 + rng.random(n)).float().to(DEV)
    top = {"labels": 0, "teacher": 3, "teacher twice": 4}[kind]
    ids = np.stack([rng.permutation(HELD)[:max(top, 1)] for _ in range(n)])
    if kind == "teacher twice":
        ids[:, 3] = ids[:, 1]
    teacher = None if top == 0 else torch.from_numpy(rng.standard_normal((n, top))).float().to(DEV)
    loss, dx, packed = torch.empty(n, device=DEV), torch.empty_like(x), torch.zeros(2 * S, dtype=packed_dt, device=DEV)
    work = rs.rs_head_workspace(plan, 0, n, top=top, packed=packed)
    if top:
        rs.rs_distill_grad(plan, 0, flat, x, torch.from_numpy(ids).to(DEV), teacher, loss, dx, packed, work, weights=weights)
    else:
        rs.rs_head_grad(plan, 0, flat, x, torch.from_numpy(ids[:, 0].copy()).to(DEV), loss, dx, packed, work, weights=weights)
    _, p, q, _ = OH.losses(x.double().cpu().numpy(), table, ids, None if teacher is None else teacher.double().cpu().numpy())
    a, size = weights.double().cpu().numpy()[:, None], np.abs(table)
    want = a * ((p - q) @ table)
    slack = a * ((2.0 ** -8 * p * (q == 0) + 100 * U * (p + q) + 16 * U * np.abs(p - q)) @ size) + 4 * U * np.abs(want)
    off = slack + _half_step(np.abs(want) + slack)
    assert (np.abs(dx.double().cpu().numpy() - want) <= off).all()
    rounded = _bf16(a * (_bf16(p - q) @ table))
    assert n == 1 or (np.abs(rounded - want) > off).mean() > 0.02
    plan.close()
