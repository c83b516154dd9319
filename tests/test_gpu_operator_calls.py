"""Calls of the embedding and matrix operators in the ways that the header
allows: captured and replayed with merges in several passes and with two-part
operands, two at once on streams of their own, ids of more than one dimension,
fewer slices than ranks, one plan's workspace for smaller calls."""
import numpy as np
import pytest
import torch

from oracle import muon as OM
from tests.test_gpu_muon import DEV, _flat, _gaussian, _get, _rel
from workloads import TensorSpec

pytestmark = pytest.mark.gpu


def _load(rs, specs, V=1, R_mat=None, **kw):
    S, starts, _, _ = rs.rs_plan_build(specs, V)
    return rs.rs_plan_load(specs, V, S, starts, R_mat, **kw)


def _sums(ids, dy, rows):
    keep = (ids >= 0) & (ids < rows)
    return torch.zeros(rows, dy.shape[1], device=DEV).index_add_(0, ids[keep], dy[keep])


@pytest.mark.parametrize("n", [40_000, 150_000])
def test_captured_gradient_with_several_merges(gpu_lib, n):
    import structure_aware_grouped_amd as rs
    rows, cols = 3001, 8
    plan = _load(rs, [TensorSpec("table", rows, cols, "ROWS", 1)])
    ids = torch.randint(0, rows, (n,), device=DEV)
    dy = torch.randint(-3, 4, (n, cols), device=DEV).float()          # whole numbers: sums are exact
    packed, work = torch.zeros(plan.S, device=DEV), rs.rs_embed_workspace(plan, 0, n)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rs.rs_embed_grad(plan, 0, ids, dy, packed, work, scale=-2.0)
    for k in range(4):
        ids.copy_(torch.randint(-1, rows // (k + 1), (n,), device=DEV))
        dy.copy_(torch.randint(-3, 4, (n, cols), device=DEV).float())
        packed.fill_(float("nan"))
        work.random_()
        torch.cuda.synchronize()
        graph.replay()
        want = _sums(ids, dy, rows) * -2.0
        torch.cuda.synchronize()
        assert torch.equal(packed[:rows * cols].view(rows, cols), want)
    del graph
    plan.close()


def test_captured_step_with_two_parts(gpu_lib):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(51)
    specs = [TensorSpec("a", 300, 200, "WHOLE"), TensorSpec("b", 64, 48, "WHOLE"), TensorSpec("c", 70, 1500, "WHOLE")]
    plan = _load(rs, specs, 3, muon_parts=2)
    grad = _flat(plan, [_gaussian(rng, sp.rows, sp.cols) for sp in specs], fill=0.0)
    par, mom, work = torch.randn_like(grad), torch.zeros_like(grad), rs.rs_muon_workspace(plan)
    ref_par, ref_mom, ref_work = par.clone(), mom.clone(), torch.empty_like(work)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rs.rs_muon_step(plan, par, grad, mom, work, lr=0.02)
    for _ in range(4):
        grad.copy_(torch.randn_like(grad) * 1e-3)
        torch.cuda.synchronize()
        graph.replay()
        rs.rs_muon_step(plan, ref_par, grad, ref_mom, ref_work, lr=0.02)
        torch.cuda.synchronize()
        assert torch.equal(par, ref_par) and torch.equal(mom, ref_mom)
    del graph
    plan.close()


def test_two_gradients_at_once_with_a_workspace_each(gpu_lib):
    import structure_aware_grouped_amd as rs
    rows, cols, n = 5000, 12, 70_000
    plan = _load(rs, [TensorSpec("a", rows, cols, "ROWS", 1), TensorSpec("b", rows, cols, "ROWS", 1)], 2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ids = [torch.randint(-1, rows, (n,), device=DEV) for _ in streams]
    dys = [torch.randint(-3, 4, (n, cols), device=DEV).float() for _ in streams]
    works = [rs.rs_embed_workspace(plan, k, n) for k in range(2)]
    packed = torch.zeros(plan.R_mat * plan.S, device=DEV)              # one buffer, two intervals
    torch.cuda.synchronize()
    for _ in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                rs.rs_embed_grad(plan, k, ids[k], dys[k], packed, works[k], prev=packed)
    torch.cuda.synchronize()
    for k in range(2):
        got = packed[plan.starts[k]:plan.starts[k] + rows * cols].view(rows, cols)
        assert torch.equal(got, _sums(ids[k], dys[k], rows) * 10)
    plan.close()


def test_ids_in_two_dimensions_and_a_larger_workspace(gpu_lib):
    import structure_aware_grouped_amd as rs
    rows, cols = 400, 24
    plan = _load(rs, [TensorSpec("table", rows, cols, "ROWS", 1)])
    flat = torch.randn(plan.S, device=DEV)
    work = rs.rs_embed_workspace(plan, 0, 50_000)
    work.random_()
    for shape in ((7, 33), (1, 1), (4, 5000), (3, 0)):
        ids = torch.randint(-2, rows + 2, shape, device=DEV, dtype=torch.int32)
        out = torch.empty(*shape, cols, device=DEV)
        rs.rs_embed_rows(plan, 0, flat, ids, out, scale=0.5)
        named = (ids >= 0) & (ids < rows)
        table = flat[:rows * cols].view(rows, cols)
        assert torch.equal(out, torch.where(named[..., None], table[ids.clamp(0, rows - 1).long()] * 0.5, 0.0))
        dy = torch.randint(-3, 4, (*shape, cols), device=DEV).float()
        packed = torch.full((plan.S,), float("nan"), device=DEV)
        rs.rs_embed_grad(plan, 0, ids, dy, packed, work)
        want = _sums(ids.reshape(-1).long(), dy.reshape(-1, cols), rows)
        assert torch.equal(packed[:rows * cols].view(rows, cols), want)
    plan.close()


def test_fewer_slices_than_ranks(gpu_lib):
    """R_mat slices are allocated and what lies behind them is not there to be touched."""
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(52)
    specs = [TensorSpec("w", 90, 140, "WHOLE"), TensorSpec("table", 50, 16, "ROWS", 1), TensorSpec("v", 64, 80, "WHOLE")]
    S, starts, _, _ = rs.rs_plan_build(specs, 2)
    plan = rs.rs_plan_load(specs, 6, S, starts, 2)
    total = plan.R_mat * S
    assert total == 2 * S
    mats = [_gaussian(rng, 90, 140), None, _gaussian(rng, 64, 80)]
    whole = torch.full((total + 4096,), 7.0, dtype=torch.bfloat16, device=DEV)
    rs.rs_orthogonalize(plan, _flat(plan, mats), whole[:total], rs.rs_muon_workspace(plan))
    for i in (0, 2):
        assert _rel(_get(plan, whole, i), OM.orthogonalize(mats[i])) <= 2.0 ** -8 + 15 ** 0.5 * 2.0 ** -11
    assert bool((whole[total:] == 7.0).all())
    ids = torch.randint(0, 50, (30,), device=DEV)
    dy = torch.randint(-3, 4, (30, 16), device=DEV).float()
    packed = torch.full((total + 4096,), 7.0, device=DEV)
    rs.rs_embed_grad(plan, 1, ids, dy, packed[:total], rs.rs_embed_workspace(plan, 1, 30))
    at = starts[1]
    assert torch.equal(packed[at:at + 800].view(50, 16), _sums(ids, dy, 50))
    assert bool((packed[:at] == 7.0).all()) and bool((packed[at + 800:] == 7.0).all())
    plan.close()
