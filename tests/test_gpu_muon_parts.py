"""rs_orthogonalize and rs_muon_step with two-part operands for every matrix
(muon_parts=2) against the Newton-Schulz iteration in 64 bits.

Tolerance, as the Frobenius norm of the difference over that of the result,
ahead of any output rounding. A two-part operand is off by at most 2^-22 of
each value (two roundings of 2^-11), the dropped low * low is at most another
2^-22 of each factor's, so 2 * 2^-22 per operand. A sum of k products in fp32
takes k - 1 additions, each off by at most 2^-24 of what it has summed so far
(in what order a matrix instruction adds its own products is not documented:
every addition counts); what it has summed so far is of the size of the result
and of the root of the sum of the products' squares, and the k roundings do not
add up in phase: sqrt(k) * 2^-24 of these sizes. How far such roundings move the result depends on the
matrix: steps raise directions far below the strongest one, and errors in them,
by up to 3.44 each. So the bound is what the iteration in 64 bits gives when
every operand and every sum is off by its largest rounding with random signs:
the largest of eight draws. Roundings spread over [-largest, largest] are
sqrt(3) smaller than that in the mean square."""
import numpy as np
import pytest
import torch

from oracle import muon as OM
from tests.test_gpu_muon import DEV, SHAPES, _flat, _gaussian, _get, _rel, _weak, tile  # noqa: F401  (a fixture)
from workloads import TensorSpec

pytestmark = pytest.mark.gpu


def tol(g, coeffs=(OM.COEFFS,) * 5, draws=8):
    """The largest relative change of the result under the largest roundings with random signs."""
    g = np.asarray(g, dtype=np.float64)
    g = g.T if g.shape[0] > g.shape[1] else g
    want, worst = OM.orthogonalize(g, coeffs), 0.0
    for seed in range(draws):
        rng = np.random.default_rng(seed)

        def sign(x):
            return rng.choice((-1.0, 1.0), x.shape)

        def off(x):
            return x * (1.0 + 2 * 2.0 ** -22 * sign(x))

        def product(x, y):
            z = off(x) @ off(y)
            return z + np.sqrt(x.shape[1]) * 2.0 ** -24 * (np.abs(z) + np.sqrt((x * x) @ (y * y))) * sign(z)

        x = g / (np.linalg.norm(g) + 1e-7)
        for a, b, c in coeffs:
            s = product(x, x.T)
            x = a * x + product(b * off(s) + c * product(s, s), x)
        worst = max(worst, _rel(x, want))
    return worst


def _load(rs, shapes):
    specs = [TensorSpec(f"w{i}", r, c, "WHOLE") for i, (r, c) in enumerate(shapes)]
    S, starts, _, _ = rs.rs_plan_build(specs, len(specs))
    return rs.rs_plan_load(specs, len(specs), S, starts, muon_parts=2)


def _bare_step(rs, plan, mats, coeffs=OM.COEFFS, steps=5):
    """The parameters after one step from zero at rate 1 on these momenta: minus the orthogonal matrices, in fp32."""
    par, mom = _flat(plan, [np.zeros_like(m) for m in mats]), _flat(plan, [np.zeros_like(m) for m in mats])
    work = rs.rs_muon_workspace(plan)
    work.fill_(0xFF)
    rs.rs_muon_step(plan, par, _flat(plan, mats), mom, work, lr=1.0, nesterov=False, update_scale="none", coeffs=coeffs,
                    steps=steps)
    return par


@pytest.mark.parametrize("make", [_gaussian, _weak])
def test_step_is_near_64_bits(gpu_lib, tile, make):  # noqa: F811
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(21)
    plan = _load(rs, SHAPES)
    mats = [make(rng, r, c) for r, c in SHAPES]
    par = _bare_step(rs, plan, mats)
    for i, g in enumerate(mats):
        err = _rel(_get(plan, par, i), -OM.orthogonalize(g))
        # and the final fp32 value, 2^-24
        assert err <= tol(g) + 2.0 ** -24, (SHAPES[i], err)
    plan.close()


def test_orthogonalize_differs_by_its_own_rounding_only(gpu_lib):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(22)
    shapes = [(300, 257), (128, 640), (1030, 1600)]
    plan = _load(rs, shapes)
    mats = [_gaussian(rng, r, c) for r, c in shapes]
    out = torch.zeros(plan.R_mat * plan.S, dtype=torch.bfloat16, device=DEV)
    rs.rs_orthogonalize(plan, _flat(plan, mats), out, rs.rs_muon_workspace(plan))
    for i, g in enumerate(mats):
        want = OM.orthogonalize(g)
        got = _get(plan, out, i)
        # half a bf16 step of each value, and the error ahead of it, which moves no value far
        slack = tol(g) * np.linalg.norm(want)
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + slack).all()
        near = torch.from_numpy(want).bfloat16().double().numpy()
        assert abs(_rel(got, want) - _rel(near, want)) <= 1e-2 * _rel(near, want)
    plan.close()


@pytest.mark.parametrize("shape", [(1030, 4100), (2100, 1500)])
def test_larger_matrices(gpu_lib, shape):
    import structure_aware_grouped_amd as rs
    from tests.test_gpu_muon import _exact_on_device
    rng = np.random.default_rng(23)
    plan = _load(rs, [shape])
    g = _weak(rng, *shape)
    par = _bare_step(rs, plan, [g])
    r, c = shape
    want = -_exact_on_device(torch.from_numpy(g).to(DEV))
    got = par[plan.starts[0]:plan.starts[0] + r * c].view(r, c).double()
    assert ((got - want).norm() / want.norm()).item() <= tol(g, draws=1) + 2.0 ** -24
    plan.close()
