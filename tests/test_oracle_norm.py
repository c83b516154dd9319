"""The layer norm oracle by hand and against differences, and the refusals of
the layer norm calls that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import norm as ON
from workloads import TensorSpec


def test_oracle_by_hand():
    x = np.array([[1.0, 3.0], [2.0, 2.0]])
    assert np.allclose(ON.norm(x, [2.0, 3.0], [10.0, 20.0], eps=0.0)[0], [8.0, 23.0])
    assert np.array_equal(ON.norm(x, [2.0, 3.0], [10.0, 20.0], eps=1.0)[1], [10.0, 20.0])
    assert np.allclose(ON.norm([[3.0, 4.0]], [1.0, 1.0], eps=0.0, center=False), np.array([[3.0, 4.0]]) / np.sqrt(12.5))


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("cols", [1, 2, 9, 40])
def test_gradients_against_differences(center, cols):
    rng = np.random.default_rng(cols)
    x, dy = rng.standard_normal((5, cols)) + 0.5, rng.standard_normal((5, cols))
    w, b = rng.standard_normal(cols), rng.standard_normal(cols)
    dx, dw, db = ON.norm_grad(x, dy, w, 1e-3, center)
    f = lambda x, w, b: (dy * ON.norm(x, w, b, 1e-3, center)).sum()  # noqa: E731
    step = 1e-5                # central differences: step^2 times a third derivative of at most about 1e3
    for _ in range(6):
        vx, vw, vb = rng.standard_normal(x.shape), rng.standard_normal(cols), rng.standard_normal(cols)
        diff = (f(x + step * vx, w + step * vw, b + step * vb) - f(x - step * vx, w - step * vw, b - step * vb)) / (2 * step)
        assert abs(diff - (dx * vx).sum() - (dw * vw).sum() - (db * vb).sum()) < 1e-6 * (1 + abs(diff))


def test_null_plans():
    from structure_aware_grouped_amd import binding as b
    lib = b.load()
    p, n = ctypes.c_void_p(1 << 20), ctypes.c_int64(7)
    assert lib.rs_layer_norm(None, 0, -1, p, 1, p, 1, 1, 1e-5, 1, p, 1, None) == b.RS_EINVAL
    assert lib.rs_layer_norm_grad(None, 0, -1, p, 1, p, 1, p, 1, 1, 1e-5, 1, p, None, p, 0, 1, 1.0, p, 64, None) == b.RS_EINVAL
    assert lib.rs_layer_norm_workspace(None, 0, 1, ctypes.byref(n)) == b.RS_EINVAL and n.value == 7


def test_binding_refuses_bad_buffers(monkeypatch):
    from structure_aware_grouped_amd import binding as b
    monkeypatch.setattr(b, "_dev_check", lambda plan, *t: None)
    plan = b.Plan.__new__(b.Plan)
    plan._h, plan.numels, plan.device, plan.R_mat, plan.S, plan.n_qblocks = None, [8, 8], 0, 1, 64, 0
    plan.specs, plan.starts, plan.V = [TensorSpec("w", 8, 1, "ROWS", 1), TensorSpec("b", 8, 1, "ROWS", 1)], [0, 16], 1
    flat, x, y, dx = torch.zeros(64), torch.zeros(3, 8), torch.zeros(3, 8), torch.zeros(3, 8)
    packed, work, half = torch.zeros(64), torch.zeros(100, dtype=torch.uint8), torch.zeros(64, dtype=torch.bfloat16)
    bad = [lambda: b.rs_layer_norm(plan, 2, flat, x, y),
           lambda: b.rs_layer_norm(plan, -1, flat, x, y),
           lambda: b.rs_layer_norm(plan, 0, flat, x, y, bias=2),
           lambda: b.rs_layer_norm(plan, 0, flat, x, y, bias=-1),
           lambda: b.rs_layer_norm(plan, 0, flat, x, y[:2]),
           lambda: b.rs_layer_norm(plan, 0, flat, x.half(), y),
           lambda: b.rs_layer_norm(plan, 0, flat[:60], x, y),
           lambda: b.rs_layer_norm(plan, 0, flat, x, x),
           lambda: b.rs_layer_norm(plan, 0, flat, torch.zeros(3, 7), y),
           lambda: b.rs_layer_norm(plan, 0, flat, x, flat[:24]),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y, dx, packed, work.float()),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y, dx.to(torch.bfloat16), packed, work),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y, dx, packed.double(), work),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y, x, packed, work),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y, y, packed, work),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y, packed[:24], packed, work),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y, dx, flat, work),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y, dx, packed, work, prev=half),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y, dx, half, work, prev=half.view(torch.float32)),
           lambda: b.rs_layer_norm_grad(plan, 0, flat, x, y[:1], dx, packed, work)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
