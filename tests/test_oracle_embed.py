"""The embedding oracle on a hand-made case, and the refusals of the embedding
calls that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import embed as OE
from workloads import TensorSpec


def test_oracle_by_hand():
    table = np.array([[1, 2], [3, 4], [5, 6]], dtype=np.float32)
    ids = np.array([2, -1, 0, 2, 3])
    assert OE.lookup(table, ids, 2.0).tolist() == [[10, 12], [0, 0], [2, 4], [10, 12], [0, 0]]
    total, size, count = OE.row_sums(np.array([[1, -1], [9, 9], [2, 2], [3, -3], [9, 9]]), ids, 3)
    assert total.tolist() == [[2, 2], [0, 0], [4, -4]]
    assert size.tolist() == [[2, 2], [0, 0], [4, 4]] and count.tolist() == [1, 0, 2]
    assert OE.sigma(1.0, True, 3) == np.float32(1 / 3) and OE.sigma(2.5, False, 3) == 2.5


def test_null_plans(monkeypatch):
    from structure_aware_grouped_amd import binding as b
    lib = b.load()
    fake, n = ctypes.c_void_p(1 << 20), ctypes.c_int64(7)
    assert lib.rs_embed_rows(None, 0, fake, 0, fake, 8, 1, 1.0, fake, 0, None) == b.RS_EINVAL
    assert lib.rs_embed_grad(None, 0, fake, 8, 1, fake, 0, None, fake, 0, 1, 1.0, fake, 0, None) == b.RS_EINVAL
    assert lib.rs_embed_workspace(None, 0, 1, ctypes.byref(n)) == b.RS_EINVAL and n.value == 7


def test_binding_refuses_bad_buffers(monkeypatch):
    from structure_aware_grouped_amd import binding
    monkeypatch.setattr(binding, "_dev_check", lambda plan, *t: None)
    plan = binding.Plan.__new__(binding.Plan)
    plan._h, plan.numels, plan.device, plan.R_mat, plan.S, plan.n_qblocks = None, [64], 0, 1, 64, 0
    plan.specs, plan.starts, plan.V = [TensorSpec("w", 8, 8, "ROWS", 1)], [0], 1
    flat, ids, rows, w = torch.zeros(64), torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), torch.zeros(100, dtype=torch.uint8)
    half = torch.zeros(64, dtype=torch.bfloat16)
    bad = [lambda: binding.rs_embed_rows(plan, 1, flat, ids, rows),
           lambda: binding.rs_embed_rows(plan, -1, flat, ids, rows),
           lambda: binding.rs_embed_rows(plan, 0, flat, ids.float(), rows),
           lambda: binding.rs_embed_rows(plan, 0, flat, ids, rows[:2]),
           lambda: binding.rs_embed_rows(plan, 0, flat, ids, rows.half()),
           lambda: binding.rs_embed_rows(plan, 0, flat[:60], ids, rows),
           lambda: binding.rs_embed_rows(plan, 0, flat.double(), ids, rows),
           lambda: binding.rs_embed_rows(plan, 0, flat, ids, flat[:24]),
           lambda: binding.rs_embed_grad(plan, 0, ids, rows, flat, w.float()),
           lambda: binding.rs_embed_grad(plan, 0, ids, rows, flat.double(), w),
           lambda: binding.rs_embed_grad(plan, 0, ids, rows.int(), flat, w),
           lambda: binding.rs_embed_grad(plan, 0, ids, flat[:24], flat, w),
           lambda: binding.rs_embed_grad(plan, 0, ids, rows, flat, w, prev=half),
           lambda: binding.rs_embed_grad(plan, 0, ids, rows, flat, w, prev=flat[:60]),
           lambda: binding.rs_embed_grad(plan, 0, ids, rows, half, w, prev=half.view(torch.float32))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
