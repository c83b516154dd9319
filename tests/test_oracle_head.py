"""The head's oracle by hand and against differences, and the refusals of the
head's calls that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import head as OH
from workloads import TensorSpec


def test_oracle_by_hand():
    x, table = np.array([[1.0], [2.0], [5.0]]), np.array([[0.0], [np.log(3.0)]])
    loss, p, full, live = OH.losses(x, table, [1, 0, -100])
    assert np.allclose(loss, [-np.log(0.75), np.log(10.0), 0.0]) and live.tolist() == [True, True, False]
    assert np.allclose(p[0], [0.25, 0.75]) and full.tolist() == [[0, 1], [1, 0], [0, 0]]
    # a teacher that says 3 : 1, once in two places that name the same row
    ids, z = [[0, 1, -1], [0, 0, 1]], np.log([[3.0, 1.0, 9.0], [1.5, 1.5, 1.0]])
    loss, p, full, _ = OH.losses(x[:2], table, ids, z)
    assert np.allclose(full, 0.25 * np.array([[3, 1], [3, 1]]))
    assert np.isclose(loss[0], 0.75 * np.log(0.75 / 0.25) + 0.25 * np.log(0.25 / 0.75))
    q, live = OH.shares([[0, 1], [5, -1], [0, 1]], 2, np.array([[-np.inf, 0.0], [1.0, 1.0], [-np.inf, -np.inf]]))
    assert q.tolist() == [[0, 1], [0, 0], [0, 0]] and live.tolist() == [True, False, False]


@pytest.mark.parametrize("top", [0, 1, 4])
def test_gradients_against_differences(top):
    rng = np.random.default_rng(top)
    n, rows, cols = 6, 11, 5
    x, table, w = rng.standard_normal((n, cols)), rng.standard_normal((rows, cols)), rng.standard_normal(n)
    ids = rng.integers(-2, rows, (n, max(top, 1)))
    teacher, T = (rng.standard_normal((n, top)), 1.7) if top else (None, 1.0)
    dx, dtable, _, _ = OH.gradients(x, table, ids, w, teacher, T, 0.75)
    f = lambda x, table: (w * OH.losses(x, table, ids, teacher, T, 0.75)[0]).sum()  # noqa: E731
    step = 1e-5
    for _ in range(6):
        vx, vt = rng.standard_normal(x.shape), rng.standard_normal(table.shape)
        diff = (f(x + step * vx, table + step * vt) - f(x - step * vx, table - step * vt)) / (2 * step)
        assert abs(diff - (dx * vx).sum() - (dtable * vt).sum()) < 1e-6 * (1 + abs(diff))


def test_null_plans():
    from structure_aware_grouped_amd import binding as b
    lib = b.load()
    p, n = ctypes.c_void_p(1 << 20), ctypes.c_int64(7)
    assert lib.rs_head_loss(None, 0, p, p, 1, p, 8, 1.0, p, 0, p, 64, None) == b.RS_EINVAL
    assert lib.rs_head_grad(None, 0, p, p, 1, p, 8, None, 1.0, p, p, None, p, 0, 1, 1.0, 0, p, 64, None) == b.RS_EINVAL
    assert lib.rs_distill_loss(None, 0, p, p, 1, p, 8, p, 0, 2, 1.0, 1.0, p, 0, p, 64, None) == b.RS_EINVAL
    assert lib.rs_distill_grad(None, 0, p, p, 1, p, 8, p, 0, 2, None, 1.0, 1.0, p, p, None, p, 0, 1, 1.0, 0, p, 64, None) == b.RS_EINVAL
    assert lib.rs_head_workspace(None, 0, 1, 0, 0, 0, 0, ctypes.byref(n)) == b.RS_EINVAL and n.value == 7


def test_binding_refuses_bad_buffers(monkeypatch):
    from structure_aware_grouped_amd import binding as b
    monkeypatch.setattr(b, "_dev_check", lambda plan, *t: None)
    plan = b.Plan.__new__(b.Plan)
    plan._h, plan.numels, plan.device, plan.R_mat, plan.S, plan.n_qblocks = None, [64], 0, 1, 64, 0
    plan.specs, plan.starts, plan.V = [TensorSpec("head", 8, 8, "ROWS", 1)], [0], 1
    flat, x, dx = (torch.zeros(n, dtype=torch.bfloat16) for n in (64, 24, 24))
    ids, loss, work = torch.zeros(3, dtype=torch.int64), torch.zeros(3), torch.zeros(99, dtype=torch.uint8)
    packed, w, tid, tl = torch.zeros(64), torch.zeros(3), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    half = torch.zeros(64, dtype=torch.bfloat16)
    bad = [lambda: b.rs_head_loss(plan, 1, flat, x, ids, loss, work),
           lambda: b.rs_head_loss(plan, 0, flat.float(), x, ids, loss, work),
           lambda: b.rs_head_loss(plan, 0, flat[:60], x, ids, loss, work),
           lambda: b.rs_head_loss(plan, 0, flat, x.float(), ids, loss, work),
           lambda: b.rs_head_loss(plan, 0, flat, x[:23], ids, loss, work),
           lambda: b.rs_head_loss(plan, 0, flat, x, ids[:2], loss, work),
           lambda: b.rs_head_loss(plan, 0, flat, x, ids.float(), loss, work),
           lambda: b.rs_head_loss(plan, 0, flat, x, ids, loss[:2], work),
           lambda: b.rs_head_loss(plan, 0, flat, x, ids, loss.double(), work),
           lambda: b.rs_head_loss(plan, 0, flat, x, ids, loss, work.float()),
           lambda: b.rs_head_loss(plan, 0, flat, x, ids, ids.view(torch.float32)[:3], work),
           lambda: b.rs_distill_loss(plan, 0, flat, x, tid, tl[:2], loss, work),
           lambda: b.rs_distill_loss(plan, 0, flat, x, tid, tl.half(), loss, work),
           lambda: b.rs_distill_loss(plan, 0, flat, x, ids, loss, loss, work),
           lambda: b.rs_distill_loss(plan, 0, flat, x, tid.view(2, 3), tl.view(2, 3), loss, work),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx[:16], packed, work),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx.float(), packed, work),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, x, packed, work),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx, packed.double(), work),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx, packed[:60], work),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx, packed, work, weights=w[:2]),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx, packed, work, weights=w.double()),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx, packed, work, weights=loss),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx, packed, work, prev=half),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx, flat, work),
           lambda: b.rs_head_grad(plan, 0, flat, x, ids, loss, dx, packed, packed.view(torch.uint8)),
           lambda: b.rs_distill_grad(plan, 0, flat, x, tid, tl, loss, dx, packed, work, weights=tl),
           lambda: b.rs_head_workspace(plan, 0, 3, packed=torch.float64)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
