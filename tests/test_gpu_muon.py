"""rs_orthogonalize and rs_muon_step against the Newton-Schulz iteration in 64
bits (oracle.muon).

Tolerance of the orthogonalised matrix, as the Frobenius norm of the
difference over that of the result: every step rounds three operands to fp16
(A, the polynomial, the high part of X in the off-diagonal product), each by
at most 2^-11 of itself, and the polynomial near the singular values that the
steps lead to (0.7 to 1.2) has slopes of about 1, so roundings neither grow nor
add up in phase: sqrt(3 * steps) * 2^-11, 1.9e-3 for five steps. The bf16
result adds its own rounding, at most 2^-8 of each value. Momentum is two fp32
operations and must agree bit for bit."""
import math

import numpy as np
import pytest
import torch

from oracle import muon as OM
from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SHAPES = [(2, 2), (2, 3), (3, 2), (2, 1000), (1000, 2), (17, 5), (48, 64), (64, 48), (64, 64), (65, 64), (63, 129),
          (64, 256), (256, 33), (64, 257), (128, 128), (129, 127), (256, 256), (257, 300), (300, 257), (333, 1001), (520, 130), (384, 640)]


def tol(steps):
    return math.sqrt(3 * steps) * 2.0 ** -11


def _load(rs, specs, V=None):
    V = len(specs) if V is None else V
    S, starts, _, _ = rs.rs_plan_build(specs, V)
    return rs.rs_plan_load(specs, V, S, starts, V, 0)


def _gaussian(rng, r, c):
    return rng.standard_normal((r, c)).astype(np.float32) * np.float32(1e-3)


def _weak(rng, r, c):
    """A few strong directions over others a hundred times weaker."""
    k = max(1, min(r, c, 16) // 2)
    low = rng.standard_normal((r, k)) @ rng.standard_normal((k, c))
    return ((low + 0.01 * rng.standard_normal((r, c))) * 1e-3).astype(np.float32)


def _flat(plan, mats, dtype=torch.float32, fill=float("nan")):
    """A flat buffer holding `mats` at the plan's starts, `fill` everywhere else."""
    flat = torch.full((plan.R_mat * plan.S,), fill, dtype=dtype, device=DEV)
    for m, at in zip(mats, plan.starts):
        if m is not None:
            flat[at:at + m.size] = torch.from_numpy(np.ascontiguousarray(m).reshape(-1)).to(DEV).to(dtype)
    return flat


def _get(plan, flat, i):
    sp, at = plan.specs[i], plan.starts[i]
    return flat[at:at + sp.rows * sp.cols].double().cpu().numpy().reshape(sp.rows, sp.cols)


def _rel(x, y):
    return np.linalg.norm(x - y) / max(np.linalg.norm(y), 1e-300)


@pytest.fixture(params=["", "64", "128", "256", "64 pairs", "128 pairs", "256 pairs"])
def tile(request, monkeypatch):
    """The output tile of the products: the plan's own choice (small matrices in one workgroup
    each), or one size for all; and the first two steps together."""
    monkeypatch.setenv("RS_MUON_TILE", request.param.split(" ")[0])
    monkeypatch.setenv("RS_MUON_PAIRS", "1" if "pairs" in request.param else "0")
    return request.param


@pytest.mark.parametrize("make", [_gaussian, _weak])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize_matches_64_bits(gpu_lib, tile, dtype, make):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(11)
    specs = [TensorSpec(f"w{i}", r, c, "WHOLE") for i, (r, c) in enumerate(SHAPES)]
    plan = _load(rs, specs)
    mats = [torch.from_numpy(make(rng, r, c)).to(dtype).double().numpy() for r, c in SHAPES]
    src = _flat(plan, mats, dtype)
    out = torch.full((plan.R_mat * plan.S,), 7.0, dtype=torch.bfloat16, device=DEV)
    work = rs.rs_muon_workspace(plan)
    work.fill_(0xFF)                       # NaN in every format: nothing may be read before it is written
    rs.rs_orthogonalize(plan, src, out, work)
    torch.cuda.synchronize()
    for i, g in enumerate(mats):
        want = OM.orthogonalize(g)
        got = _get(plan, out, i)
        assert _rel(got, want) <= math.hypot(tol(5), 2.0 ** -8), (SHAPES[i], _rel(got, want))
    inside = torch.zeros(out.numel(), dtype=torch.bool, device=DEV)
    for sp, at in zip(specs, plan.starts):
        inside[at:at + sp.rows * sp.cols] = True
    assert bool((out[~inside] == 7.0).all())
    first = out.clone()
    rs.rs_orthogonalize(plan, src, out, work)
    assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    plan.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nesterov,scale_mode,wd", [(True, "rms", 0.1), (False, "spectral", 0.0), (True, "none", 0.01)])
def test_muon_step_matches_64_bits(gpu_lib, tile, dtype, nesterov, scale_mode, wd):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(12)
    specs = [TensorSpec(f"w{i}", r, c, "WHOLE") for i, (r, c) in enumerate(SHAPES)]
    plan = _load(rs, specs)
    lr, mu = 0.5, 0.95                     # a rate at which the update is as large as the parameters
    grads = [torch.from_numpy(_weak(rng, r, c)).to(dtype).float().numpy() for r, c in SHAPES]
    moms = [_gaussian(rng, r, c) * 10 for r, c in SHAPES]
    pars = [_gaussian(rng, r, c) * 20 for r, c in SHAPES]
    grad, mom, par = _flat(plan, grads, dtype), _flat(plan, moms), _flat(plan, pars)
    work = rs.rs_muon_workspace(plan)
    work.fill_(0xFF)
    for _ in range(2):                     # two steps: the second starts from the first one's state
        rs.rs_muon_step(plan, par, grad, mom, work, lr=lr, momentum_decay=mu, weight_decay=wd, nesterov=nesterov,
                        update_scale=scale_mode)
        torch.cuda.synchronize()
        for i, (r, c) in enumerate(SHAPES):
            moms[i] = OM.momentum_f32(moms[i], grads[i], mu)
            assert np.array_equal(_get(plan, mom, i).astype(np.float32), moms[i]), SHAPES[i]
            update = lr * OM.update_scale(scale_mode, r, c) * OM.orthogonalize(
                OM.muon_direction(moms[i], grads[i], mu, nesterov))
            want = (1.0 - np.float64(np.float32(lr)) * np.float64(np.float32(wd))) * pars[i].astype(np.float64) - update
            got = _get(plan, par, i)
            # the update's error, and three fp32 roundings of each value
            bound = tol(5) * np.linalg.norm(update) + 3 * 2.0 ** -24 * (np.linalg.norm(want) + np.linalg.norm(update))
            assert np.linalg.norm(got - want) <= bound, (SHAPES[i], np.linalg.norm(got - want) / bound)
            pars[i] = got.astype(np.float32)
    for flat in (par, mom):                # the padding's NaN is still there
        outside = torch.ones(flat.numel(), dtype=torch.bool, device=DEV)
        for sp, at in zip(specs, plan.starts):
            outside[at:at + sp.rows * sp.cols] = False
        assert bool(torch.isnan(flat[outside]).all())
    plan.close()


def test_steps_and_coefficients_per_step(gpu_lib, tile):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(13)
    specs = [TensorSpec("a", 70, 200, "WHOLE"), TensorSpec("b", 200, 70, "WHOLE")]
    plan = _load(rs, specs)
    mats = [_gaussian(rng, sp.rows, sp.cols) for sp in specs]
    src, work = _flat(plan, mats), rs.rs_muon_workspace(plan)
    out = torch.zeros(plan.R_mat * plan.S, dtype=torch.bfloat16, device=DEV)
    for coeffs in ([(1.5, -0.5, 0.0)], [(1.5, -0.5, 0.0)] * 2, [(2.0, -1.5, 0.5)] * 3, [(4.5, -6.0, 2.5), (1.5, -0.5, 0.0)], [(3.4445, -4.775, 2.0315)] * 3 + [(1.875, -1.25, 0.375)] * 3):
        rs.rs_orthogonalize(plan, src, out, work, coeffs=coeffs, steps=len(coeffs))
        for i, g in enumerate(mats):
            want = OM.orthogonalize(g, [tuple(float(np.float32(v)) for v in r) for r in coeffs])
            assert _rel(_get(plan, out, i), want) <= math.hypot(tol(len(coeffs)), 2.0 ** -8)
    plan.close()


def test_other_tensors_and_padding_are_left_alone(gpu_lib):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(14)
    specs = [TensorSpec("rows", 40, 24, "ROWS", 1), TensorSpec("w", 30, 50, "WHOLE"), TensorSpec("vec", 77, 1, "WHOLE"),
             TensorSpec("tile", 33, 40, "TILE", 16, 16), TensorSpec("row", 1, 99, "WHOLE")]
    plan = _load(rs, specs, 3)
    g = _gaussian(rng, 30, 50)
    grad = _flat(plan, [None, g, None, None, None])
    mom = _flat(plan, [None, g, None, None, None], fill=3.0)
    par = _flat(plan, [None, g, None, None, None], fill=5.0)
    rs.rs_muon_step(plan, par, grad, mom, rs.rs_muon_workspace(plan), lr=0.1)
    torch.cuda.synchronize()
    inside = torch.zeros(par.numel(), dtype=torch.bool, device=DEV)
    inside[plan.starts[1]:plan.starts[1] + 1500] = True
    assert bool((par[~inside] == 5.0).all()) and bool((mom[~inside] == 3.0).all())
    assert bool(torch.isfinite(par[inside]).all()) and not bool((par[inside] == 5.0).any())
    plan.close()
    none = _load(rs, [specs[0]], 1)        # a plan without matrices: nothing to do
    flat = torch.ones(none.R_mat * none.S, device=DEV)
    rs.rs_muon_step(none, flat, flat.clone(), flat.clone(), rs.rs_muon_workspace(none), lr=0.1)
    assert bool((flat == 1.0).all())
    none.close()


def test_zero_huge_tiny_and_non_finite_matrices(gpu_lib, tile):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(15)
    specs = [TensorSpec(f"w{i}", 40 + i, 60 - i, "WHOLE") for i in range(6)]
    plan = _load(rs, specs)
    base = [_gaussian(rng, sp.rows, sp.cols) for sp in specs]
    mats = [base[0] * 0, base[1] * np.float32(1e30), base[2] * np.float32(1e-30), base[3].copy(), base[4].copy(), base[5]]
    mats[3][5, 7] = np.nan
    mats[4][39, 55] = -np.inf
    out = torch.zeros(plan.R_mat * plan.S, dtype=torch.bfloat16, device=DEV)
    rs.rs_orthogonalize(plan, _flat(plan, mats), out, rs.rs_muon_workspace(plan), eps=1e-38)
    got = [_get(plan, out, i) for i in range(6)]
    assert not got[0].any()
    for i in (1, 2, 5):
        assert _rel(got[i], OM.orthogonalize(mats[i], eps=1e-38)) <= math.hypot(tol(5), 2.0 ** -8), i
    assert np.isnan(got[3]).all() and np.isnan(got[4]).all()
    plan.close()


def test_captured_step_replays_like_the_eager_one(gpu_lib):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(16)
    specs = [TensorSpec("a", 300, 200, "WHOLE"), TensorSpec("b", 64, 48, "WHOLE")]
    plan, other = _load(rs, specs), _load(rs, specs)
    grad = _flat(plan, [_gaussian(rng, sp.rows, sp.cols) for sp in specs], fill=0.0)
    par, mom = torch.randn_like(grad), torch.zeros_like(grad)
    out = torch.zeros(grad.numel(), dtype=torch.bfloat16, device=DEV)
    work, work2 = rs.rs_muon_workspace(plan), rs.rs_muon_workspace(plan)
    ref_par, ref_mom, ref_out = par.clone(), mom.clone(), out.clone()

    def step(pl, p, m, o, w):
        rs.rs_muon_step(pl, p, grad, m, w, lr=0.02)
        rs.rs_orthogonalize(pl, m, o, w)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):          # nothing has to run before the capture: no pointer table
        step(plan, par, mom, out, work)
    for _ in range(3):
        grad.copy_(torch.randn_like(grad) * 1e-3)
        torch.cuda.synchronize()
        graph.replay()
        step(other, ref_par, ref_mom, ref_out, work2)
        torch.cuda.synchronize()
        assert torch.equal(par, ref_par) and torch.equal(mom, ref_mom) and torch.equal(out, ref_out)
    del graph
    plan.close()
    other.close()


def test_another_stream(gpu_lib):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(17)
    specs = [TensorSpec("a", 130, 260, "WHOLE")]
    plan = _load(rs, specs)
    src, work = _flat(plan, [_gaussian(rng, 130, 260)]), rs.rs_muon_workspace(plan)
    out = torch.zeros(plan.R_mat * plan.S, dtype=torch.bfloat16, device=DEV)
    rs.rs_orthogonalize(plan, src, out, work)
    again = torch.zeros_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rs.rs_orthogonalize(plan, src, again, work)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, again)
    plan.close()


def test_calls_that_are_refused(gpu_lib):
    import structure_aware_grouped_amd as rs
    from structure_aware_grouped_amd import binding as b
    plan = _load(rs, [TensorSpec("a", 100, 300, "WHOLE")])
    n = plan.R_mat * plan.S
    src, work = torch.zeros(n, device=DEV), rs.rs_muon_workspace(plan)
    out = torch.zeros(n, dtype=torch.bfloat16, device=DEV)

    def status(fn):
        with pytest.raises(rs.RsError) as e:
            fn()
        return e.value.status

    for kw in ({"steps": 0}, {"steps": 33}, {"eps": -1.0}, {"eps": float("nan")}, {"coeffs": (1.0, float("inf"), 0.0)}):
        assert status(lambda: rs.rs_orthogonalize(plan, src, out, work, **kw)) == b.RS_EINVAL
    m, p = torch.zeros_like(src), torch.zeros_like(src)
    for kw in ({"lr": float("nan")}, {"lr": 1.0, "momentum_decay": 1.0}, {"lr": 1.0, "momentum_decay": -0.1},
               {"lr": 1.0, "weight_decay": float("inf")}):
        assert status(lambda: rs.rs_muon_step(plan, p, src, m, work, **kw)) == b.RS_EINVAL
    lib = b.load()
    c = b._coeffs(rs.MUON_COEFFS, 5)
    args = (src.data_ptr(), 0, out.data_ptr(), c, 5, 1e-7)
    assert lib.rs_orthogonalize(plan.handle, *args, work.data_ptr(), work.numel() - 1, None) == b.RS_EINVAL
    assert lib.rs_orthogonalize(plan.handle, *args, work.data_ptr() + 8, work.numel(), None) == b.RS_EALIGN
    assert lib.rs_orthogonalize(plan.handle, src.data_ptr(), b.RS_I8, out.data_ptr(), c, 5, 1e-7, work.data_ptr(),
                                work.numel(), None) == b.RS_EDTYPE
    torch.cuda.synchronize()
    assert not out.any()
    plan.close()


def _exact_on_device(g):
    x = g.double()
    x = x.T.contiguous() if x.shape[0] > x.shape[1] else x
    x = x / (x.square().sum().sqrt() + 1e-7)
    for a, b, c in (OM.COEFFS,) * 5:
        s = torch.mm(x, x.T.contiguous())
        x = a * x + torch.mm(b * s + c * torch.mm(s, s), x)
    return x.T if g.shape[0] > g.shape[1] else x


@pytest.mark.parametrize("shapes", [[(4100, 5300)], [(2050, 4100), (1031, 4097), (700, 300), (50, 60)], [(6001, 5900)],
                                    [(3000, 1100)] * 5 + [(40, 3000)]])
def test_the_plans_own_choice_at_larger_sizes(gpu_lib, shapes):
    """256-wide tiles, cut tiles and joins, the first two steps together, single- and two-part
    matrices and small ones in one group, against torch's products in 64 bits."""
    import structure_aware_grouped_amd as rs
    torch.manual_seed(18)
    plan = _load(rs, [TensorSpec(f"w{i}", r, c, "WHOLE") for i, (r, c) in enumerate(shapes)])
    src = torch.full((plan.R_mat * plan.S,), float("nan"), device=DEV)
    for (r, c), at in zip(shapes, plan.starts):
        low = torch.randn(r, 8, device=DEV) @ torch.randn(8, c, device=DEV)
        src[at:at + r * c] = (low + torch.randn(r, c, device=DEV)).reshape(-1) * 1e-3
    out = torch.zeros(src.numel(), dtype=torch.bfloat16, device=DEV)
    work = rs.rs_muon_workspace(plan)
    work.fill_(0xFF)
    rs.rs_orthogonalize(plan, src, out, work)
    for (r, c), at in zip(shapes, plan.starts):
        want = _exact_on_device(src[at:at + r * c].view(r, c))
        got = out[at:at + r * c].view(r, c).double()
        assert ((got - want).norm() / want.norm()).item() <= math.hypot(tol(5), 2.0 ** -8), (r, c)
    plan.close()


def test_two_calls_at_once_with_a_workspace_each(gpu_lib):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(19)
    specs = [TensorSpec("a", 700, 900, "WHOLE"), TensorSpec("b", 100, 50, "WHOLE")]
    plan = _load(rs, specs)
    srcs = [_flat(plan, [_gaussian(rng, sp.rows, sp.cols) for sp in specs], fill=0.0) for _ in range(2)]
    want = [torch.zeros(s.numel(), dtype=torch.bfloat16, device=DEV) for s in srcs]
    works = [rs.rs_muon_workspace(plan) for _ in srcs]
    for s, o in zip(srcs, want):
        rs.rs_orthogonalize(plan, s, o, works[0])
    torch.cuda.synchronize()
    got = [torch.zeros_like(o) for o in want]
    streams = [torch.cuda.Stream() for _ in srcs]
    for _ in range(5):
        for s, o, w, st in zip(srcs, got, works, streams):
            with torch.cuda.stream(st):
                rs.rs_orthogonalize(plan, s, o, w)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    plan.close()
