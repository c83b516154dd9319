"""The bits of table rows that no token names: +0.0, or prev + 0.0 (so +0.0
where prev is -0.0), whichever pass writes them. Below half as many tokens as
rows it is the fill, from there on the pass over the whole table."""
import numpy as np
import pytest
import torch

from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("cols", [16, 7])
@pytest.mark.parametrize("packed_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_prev", [False, True])
@pytest.mark.parametrize("scale", [-3.0, 3.0, -0.0])
@pytest.mark.parametrize("n", [0, 1, 99, 100, 101, 300])
def test_rows_without_a_token_are_plus_zero(gpu_lib, cols, packed_dt, with_prev, scale, n):
    import structure_aware_grouped_amd as rs
    rows = 200                       # the pass over the whole table from 100 tokens on
    specs = [TensorSpec("table", rows, cols, "ROWS", 1)]
    S, starts, _, _ = rs.rs_plan_build(specs, 1)
    plan = rs.rs_plan_load(specs, 1, S, starts)
    rng = np.random.default_rng(n)
    named = rng.choice(rows, 20, replace=False)
    ids = torch.from_numpy(rng.choice(named, n)).to(DEV) if n else torch.empty(0, dtype=torch.int64, device=DEV)
    dy = torch.ones(n, cols, device=DEV)
    prev = torch.full((S,), -0.0, device=DEV) if with_prev else None
    packed = torch.full((S,), float("nan"), dtype=packed_dt, device=DEV)
    rs.rs_embed_grad(plan, 0, ids, dy, packed, rs.rs_embed_workspace(plan, 0, n), prev=prev, scale=scale)
    got = packed[:rows * cols].float().view(rows, cols).cpu().numpy()
    count = np.bincount(ids.cpu().numpy(), minlength=rows).astype(np.float32)
    assert not got[count == 0].view(np.uint32).any()
    want = np.float32(scale) * count[:, None] + (np.float32(-0.0) if with_prev else np.float32(0.0) * 0)
    want = torch.from_numpy(np.ascontiguousarray(np.broadcast_to(want, got.shape))).to(packed_dt).float().numpy()
    assert np.array_equal(got[count > 0], want[count > 0])
    plan.close()
