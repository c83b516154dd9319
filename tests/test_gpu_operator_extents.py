"""The embedding and matrix operators at the ends of their ranges: offsets past
2^32, sides of 2^20, hundreds of matrices in one plan, an eps far above the
norm."""
import math

import numpy as np
import pytest
import torch

from oracle import muon as OM
from tests.test_gpu_muon import DEV, _exact_on_device, _flat, _get, _rel, tol as one_part
from workloads import TensorSpec

pytestmark = pytest.mark.gpu


def _load(rs, specs, V=1, **kw):
    S, starts, _, _ = rs.rs_plan_build(specs, V)
    return rs.rs_plan_load(specs, V, S, starts, **kw)


def test_a_table_of_more_than_2_to_32_elements(gpu_lib):
    """Rows on both sides of element 2^32 (bytes 2^33 of the gathered and 2^34 of the packed buffer)."""
    import structure_aware_grouped_amd as rs
    rows, cols, n = 70001, 61448, 96                       # 4.30e9 elements; 2^32 lies in row 69895
    plan = _load(rs, [TensorSpec("table", rows, cols, "ROWS", 1)])
    mark = torch.tensor([0, 1, 34947, 69894, 69895, 69896, rows - 2, rows - 1], device=DEV)
    gathered = torch.zeros(plan.S, dtype=torch.bfloat16, device=DEV)
    table = gathered[:rows * cols].view(rows, cols)
    table[mark] = torch.randint(-100, 101, (mark.numel(), cols), device=DEV).to(torch.bfloat16)
    ids = mark[torch.randint(0, mark.numel(), (n,), device=DEV)]
    ids[5] = -1
    out = torch.full((n, cols), float("nan"), dtype=torch.bfloat16, device=DEV)
    rs.rs_embed_rows(plan, 0, gathered, ids, out, scale=2.0)
    want = torch.stack([table[int(r)] * 2.0 if r >= 0 else torch.zeros(cols, dtype=torch.bfloat16, device=DEV) for r in ids.tolist()])
    assert torch.equal(out, want)
    dy = torch.randint(-3, 4, (n, cols), device=DEV).float()
    packed = torch.full((plan.S,), float("nan"), device=DEV)
    work = rs.rs_embed_workspace(plan, 0, n)
    view = packed[:rows * cols].view(rows, cols)
    sums = {int(r): dy[ids == r].sum(0) for r in mark.tolist()}
    for times in (1, 2):                                   # written, then added in place
        rs.rs_embed_grad(plan, 0, ids, dy, packed, work, prev=packed if times == 2 else None)
        for r, s in sums.items():
            assert torch.equal(view[r], s * times), r
            view[r] = 0.0
        assert not bool(view[:35000].any()) and not bool(view[35000:].any())      # NaN counts as true
        for r, s in sums.items():
            view[r] = s
    assert bool(torch.isnan(packed[rows * cols:]).all())
    plan.close()


@pytest.mark.parametrize("shape,dtype", [((40000, 56001), torch.bfloat16), ((66000, 33000), torch.float32)])
def test_a_matrix_of_more_than_2_to_31_elements(gpu_lib, shape, dtype):
    """One value per row or column, so that the result is the polynomials' of one number each, in place."""
    import structure_aware_grouped_amd as rs
    r, c = shape
    m, n = min(shape), max(shape)
    plan = _load(rs, [TensorSpec("w", r, c, "WHOLE")])
    src = torch.zeros(plan.S, dtype=dtype, device=DEV)
    i = torch.arange(m, device=DEV)
    j = (i * 7919 + 13) % n                                # 7919 shares no factor with either n: all different
    at = i * c + j if r <= c else j * c + i
    value = (1 + (i % 3)).to(dtype)
    src[at] = value
    out = torch.full((plan.S,), 7.0, dtype=torch.bfloat16, device=DEV)
    work = rs.rs_muon_workspace(plan)
    coeffs = [(3.4445, -4.775, 2.0315), (4.0, -6.5, 3.0)]
    rs.rs_orthogonalize(plan, src, out, work, coeffs=coeffs, steps=2)
    del work
    x = value.double() / (value.double().square().sum().sqrt() + 1e-7)
    for a, b, d in coeffs:
        x = a * x + b * x ** 3 + d * x ** 5
    got = out[at].double()
    assert bool(((got - x).abs() <= (2.0 ** -8 + one_part(2)) * x).all())
    out[at] = 0.0
    for k in range(0, r * c, 1 << 30):
        assert not bool(out[k:min(k + (1 << 30), r * c)].any())
    assert bool((out[r * c:] == 7.0).all())
    plan.close()


@pytest.mark.parametrize("shape", [(2, 2 ** 20), (2 ** 20, 3), (50, 2 ** 20), (2 ** 20, 100)])
def test_sides_of_2_to_20(gpu_lib, shape):
    import structure_aware_grouped_amd as rs
    torch.manual_seed(41)
    r, c = shape
    plan = _load(rs, [TensorSpec("w", r, c, "WHOLE")])
    g = torch.randn(r, c, device=DEV) * 1e-3
    grad, mom, par = (torch.zeros(plan.S, device=DEV) for _ in range(3))
    grad[:r * c] = g.reshape(-1)
    rs.rs_muon_step(plan, par, grad, mom, rs.rs_muon_workspace(plan), lr=1.0, nesterov=False, update_scale="none")
    want = -_exact_on_device(g)
    got = par[:r * c].view(r, c).double()
    # sums of 2^20 products: sqrt(2^20) * 2^-24 beside the operands' roundings
    assert ((got - want).norm() / want.norm()).item() <= one_part(5) + math.sqrt(15) * 2.0 ** -14
    plan.close()


def test_hundreds_of_matrices(gpu_lib):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(42)
    shapes = [tuple(int(v) for v in rng.integers(2, 90, 2)) for _ in range(700)] + [(200, 70), (1, 9), (9, 1)]
    plan = _load(rs, [TensorSpec(f"w{i}", a, b, "WHOLE") for i, (a, b) in enumerate(shapes)], 5)
    mats = [(rng.standard_normal(s) * 1e-3).astype(np.float32) for s in shapes]
    out = torch.full((plan.R_mat * plan.S,), 7.0, dtype=torch.bfloat16, device=DEV)
    rs.rs_orthogonalize(plan, _flat(plan, mats), out, rs.rs_muon_workspace(plan))
    for i, g in enumerate(mats):
        if min(g.shape) > 1:
            assert _rel(_get(plan, out, i), OM.orthogonalize(g)) <= math.hypot(one_part(5), 2.0 ** -8), g.shape
        else:
            assert (_get(plan, out, i) == 7.0).all()
    plan.close()


@pytest.mark.parametrize("shape", [(40, 60), (90, 300), (700, 500)])
@pytest.mark.parametrize("eps", [1e-3, 10.0])
def test_an_eps_far_above_the_norm(gpu_lib, shape, eps):
    """X starts 1e3 or 1e7 times too small: the steps only multiply, and the result keeps its digits."""
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(43)
    g = rng.standard_normal(shape)
    g = (g / np.linalg.norm(g) * 1e-6).astype(np.float32)
    plan = _load(rs, [TensorSpec("w", *shape, "WHOLE")])
    out = torch.zeros(plan.S, dtype=torch.bfloat16, device=DEV)
    rs.rs_orthogonalize(plan, _flat(plan, [g]), out, rs.rs_muon_workspace(plan), eps=eps)
    want = OM.orthogonalize(g, eps=eps)
    assert _rel(_get(plan, out, 0), want) <= math.hypot(one_part(5), 2.0 ** -8)
    plan.close()
