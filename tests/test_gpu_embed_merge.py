"""rs_embed_grad with more tokens than one merge takes (16 runs of 2048): two,
three and four passes over the sorted lists, the last list short or of one
token. Sums of small whole numbers are exact, so every token has to be counted
once and in its own row. And the time stays in proportion to the tokens."""
import numpy as np
import pytest
import torch

from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
RUN = 2048


def _plan(rs, rows, cols):
    specs = [TensorSpec("table", rows, cols, "ROWS", 1)]
    S, starts, _, _ = rs.rs_plan_build(specs, 1)
    return rs.rs_plan_load(specs, 1, S, starts)


@pytest.mark.parametrize("n", [16 * RUN, 16 * RUN + 1, 17 * RUN, 64 * RUN, 64 * RUN + 1, 65 * RUN - 5, 200_003, 512 * RUN + 77])
@pytest.mark.parametrize("kind", ["uniform", "power", "few", "same", "rising", "falling"])
def test_every_token_once(gpu_lib, n, kind):
    import structure_aware_grouped_amd as rs
    rows, cols = 5003, 4
    plan = _plan(rs, rows, cols)
    gen = torch.Generator(device=DEV).manual_seed(n)
    u = torch.rand(n, device=DEV, generator=gen, dtype=torch.float64)
    at = torch.arange(n, device=DEV)
    ids = {"uniform": (u * (rows + 200)).long() - 100,          # some name no row, on both sides
           "power": (rows ** u - 1).long(), "few": (u * 3).long() * 2000, "same": torch.full_like(at, 4321),
           "rising": at * rows // n, "falling": rows - 1 - at * rows // n}[kind]
    dy = torch.randint(-3, 4, (n, cols), device=DEV, generator=gen).float()
    packed = torch.full((plan.S,), 5.0, device=DEV)
    work = rs.rs_embed_workspace(plan, 0, n)
    work.fill_(0xFF)
    rs.rs_embed_grad(plan, 0, ids, dy, packed, work, prev=packed)
    keep = (ids >= 0) & (ids < rows)
    want = torch.zeros(rows, cols, dtype=torch.int64, device=DEV).index_add_(0, ids[keep], dy[keep].long())
    assert want.abs().max().item() < 2 ** 23
    assert torch.equal(packed[:rows * cols].view(rows, cols).long(), want + 5)
    first = packed.clone()
    packed.fill_(5.0)
    rs.rs_embed_grad(plan, 0, ids, dy, packed, work, prev=packed)
    assert torch.equal(packed, first)
    plan.close()


def test_time_in_proportion_to_the_tokens(gpu_lib):
    """Eight times the tokens in at most sixteen times the time (merging all runs for every token took 31)."""
    import structure_aware_grouped_amd as rs
    plan = _plan(rs, 131072, 64)
    times = []
    for n in (1 << 17, 1 << 20):
        ids = torch.randint(0, 131072, (n,), device=DEV)
        dy, packed = torch.ones(n, 64, device=DEV), torch.zeros(plan.S, device=DEV)
        work, best = rs.rs_embed_workspace(plan, 0, n), float("inf")
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            rs.rs_embed_grad(plan, 0, ids, dy, packed, work, prev=packed)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert times[1] <= 16 * times[0], times
    plan.close()
