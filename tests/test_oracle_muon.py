"""The Newton-Schulz oracle against the singular value decomposition, and the
refusals of the matrix calls that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import muon as OM
from workloads import TensorSpec


@pytest.mark.parametrize("shape", [(2, 2), (3, 7), (7, 3), (20, 20), (1, 5)])
def test_oracle_maps_singular_values_by_the_polynomial(shape):
    g = np.random.default_rng(5).standard_normal(shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.linalg.norm(g) + 1e-7)
    for a, b, c in (OM.COEFFS,) * 5:
        s = a * s + b * s ** 3 + c * s ** 5
    # the iteration works on X of norm 1 with products of norm at most a few: 1e-12 is 1e4 roundings
    assert np.abs(OM.orthogonalize(g) - (u * s) @ vt).max() < 1e-12


def test_only_whole_tensors_of_two_dimensions_are_matrices():
    assert OM.is_matrix(TensorSpec("w", 2, 2, "WHOLE"))
    for sp in (TensorSpec("v", 9, 1, "WHOLE"), TensorSpec("r", 1, 9, "WHOLE"), TensorSpec("t", 9, 9, "ROWS", 1)):
        assert not OM.is_matrix(sp)


@pytest.fixture(scope="module")
def lib():
    from structure_aware_grouped_amd import binding
    return binding.load()


def _stand_in(need):
    """A plan object that no device knows, whose workspace query says `need` bytes."""
    from structure_aware_grouped_amd import binding
    plan = binding.Plan.__new__(binding.Plan)
    plan._h, plan.numels, plan.device, plan.R_mat, plan.S, plan.n_qblocks = None, [64], 0, 1, 64, 0
    plan.specs, plan.starts = [TensorSpec("w", 8, 8, "WHOLE")], [0]
    return plan


@pytest.fixture
def binding(lib, monkeypatch):
    from structure_aware_grouped_amd import binding
    monkeypatch.setattr(binding, "_dev_check", lambda plan, *t: None)
    monkeypatch.setattr(binding, "_muon_bytes", lambda plan: 1000)
    return binding


def test_null_plans_and_arguments(lib):
    from structure_aware_grouped_amd import binding as b
    n = ctypes.c_int64(7)
    fake = ctypes.c_void_p(1 << 20)
    c = (ctypes.c_float * 15)()
    assert lib.rs_muon_workspace(None, ctypes.byref(n)) == b.RS_EINVAL and n.value == 7
    assert lib.rs_orthogonalize(None, fake, 0, fake, c, 5, 0.0, fake, 0, None) == b.RS_EINVAL
    hp = b.MuonHParamsC(0.1, 0.9, 0.0, 1e-7, 5, 1, 0)
    assert lib.rs_muon_step(None, fake, fake, 0, fake, ctypes.byref(hp), c, fake, 0, None) == b.RS_EINVAL
    assert "null plan" in lib.rs_last_error().decode()


def test_binding_refuses_bad_buffers(binding):
    plan = _stand_in(1000)
    f, h, w = torch.zeros(64), torch.zeros(64, dtype=torch.bfloat16), torch.zeros(1000, dtype=torch.uint8)
    bad = [lambda: binding.rs_orthogonalize(plan, f.half(), h, w),
           lambda: binding.rs_orthogonalize(plan, f, f.clone(), w),
           lambda: binding.rs_orthogonalize(plan, f[:63], h, w),
           lambda: binding.rs_orthogonalize(plan, f, h[:63], w),
           lambda: binding.rs_orthogonalize(plan, f, h, w[:999]),
           lambda: binding.rs_orthogonalize(plan, f, h, torch.zeros(250)),
           lambda: binding.rs_orthogonalize(plan, h, h, w),
           lambda: binding.rs_muon_step(plan, h, f, f.clone(), w, lr=0.1),
           lambda: binding.rs_muon_step(plan, f, f.double(), f.clone(), w, lr=0.1),
           lambda: binding.rs_muon_step(plan, f, f.clone(), h, w, lr=0.1),
           lambda: binding.rs_muon_step(plan, f, f, f.clone(), w, lr=0.1),
           lambda: binding.rs_muon_step(plan, f, f.clone(), f, w, lr=0.1),
           lambda: binding.rs_muon_step(plan, f, f.clone(), f.clone(), w, lr=0.1, update_scale="adam")]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    one = torch.zeros(130)
    with pytest.raises(ValueError, match="overlap"):
        binding.rs_muon_step(plan, one[:64], one[63:127], f, w, lr=0.1)


def test_coefficients_are_one_triple_or_one_per_step():
    from structure_aware_grouped_amd import binding as b
    assert list(b._coeffs((1, 2, 3), 2)) == [1, 2, 3, 1, 2, 3]
    assert list(b._coeffs([(1, 2, 3), (4, 5, 6)], 2)) == [1, 2, 3, 4, 5, 6]
    for bad, steps in (([(1, 2, 3)], 2), ((1, 2), 1), ([(1, 2, 3), (1, 2)], 2), ([], 1)):
        with pytest.raises(ValueError):
            b._coeffs(bad, steps)
