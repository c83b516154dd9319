"""The operators of one training step together, on one plan's flat buffers: an
embedding lookup from the gathered buffer, a small network in torch, its
gradients packed (the table's by rs_embed_grad beside its dense one from the
tied output, the others' by rs_pack_scatter), the Muon step on the matrices and
the 8-bit AdamW step on the rest. Against the same steps in plain torch and the
oracles; and every quantisation block, matrix and table keeps its own values."""
import os
import re
import textwrap

import numpy as np
import pytest
import torch

from oracle import adam as OA, muon as OM
from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_embedding_network_and_optimiser_steps(gpu_lib):
    import structure_aware_grouped_amd as rs
    torch.manual_seed(3)
    vocab, d, h, n, V, lr = 300, 96, 160, 200, 4, 0.05
    specs = [TensorSpec("table", vocab, d, "TILE", 32, 32), TensorSpec("w1", h, d, "WHOLE"), TensorSpec("w2", d, h, "WHOLE"),
             TensorSpec("norm", d, 1, "FLAT", 64)]
    S, starts, _, _ = rs.rs_plan_build(specs, V)
    plan = rs.rs_plan_load(specs, V, S, starts, V, 0)
    total = V * S
    param = torch.zeros(total, device=DEV)

    def view(flat, i):
        sp = specs[i]
        return flat[starts[i]:starts[i] + sp.rows * sp.cols].view(sp.rows, sp.cols)

    for i, scale in enumerate((1.0, 0.1, 0.1, 1.0)):
        view(param, i).copy_(torch.randn(specs[i].rows, specs[i].cols, device=DEV) * scale)
    momentum, packed = torch.zeros(total, device=DEV), torch.zeros(total, device=DEV)
    codes = [torch.zeros(total, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.ones(plan.n_qblocks, device=DEV) for _ in range(2)]
    work, mwork = rs.rs_embed_workspace(plan, 0, n), rs.rs_muon_workspace(plan)

    for step in range(1, 4):
        ids = torch.randint(-1, vocab, (n,), device=DEV)
        target = torch.randint(0, vocab, (n,), device=DEV)
        gathered = param.clone()                       # what an all-gather would give
        x = torch.empty(n, d, device=DEV)
        rs.rs_embed_rows(plan, 0, gathered, ids, x, scale=2.0)
        leaves = [view(gathered, i).clone().requires_grad_() for i in range(4)]
        xin = x.clone().requires_grad_()

        def loss_of(table_in, leaves):
            y = torch.nn.functional.silu(table_in @ leaves[1].T) @ leaves[2].T
            y = (table_in + y) * leaves[3].view(1, d)
            return torch.nn.functional.cross_entropy(y @ leaves[0].T, target)   # the output is tied to the table

        loss_of(xin, leaves).backward()
        rs.rs_pack_scatter(plan, [l.grad.contiguous() for l in leaves], packed)
        rs.rs_embed_grad(plan, 0, ids, xin.grad, packed, work, prev=packed, scale=2.0, inv_v=True)

        # the same gradients by torch alone
        plain = [view(gathered, i).clone().requires_grad_() for i in range(4)]
        named = ids >= 0
        loss_of(torch.where(named[:, None], plain[0][ids.clamp(min=0)] * 2.0, 0.0), plain).backward()
        for i in range(4):
            want = plain[i].grad / V
            got = view(packed, i)
            # fp32 sums of up to n terms in another order, on either side
            assert (got - want).norm() <= 2 * n * 2.0 ** -24 * want.norm() + 1e-12, (step, i)

        before, mom_before, grad = param.clone(), momentum.clone(), packed.clone()
        rs.rs_muon_step(plan, param, packed, momentum, mwork, lr=lr, weight_decay=0.1)
        state = [t.cpu().numpy().copy() for t in (codes[0], scales[0], codes[1], scales[1])]
        hyper = OA.AdamHyper(1e-3, 0.9, 0.99, 1e-8, 0.0, step)
        rs.rs_adam8_step(plan, param, packed, codes[0], scales[0], codes[1], scales[1], 1e-3, 0.9, 0.99, 1e-8, 0.0, step)
        torch.cuda.synchronize()
        for i in (1, 2):
            m = OM.momentum_f32(view(mom_before, i).cpu().numpy(), view(grad, i).cpu().numpy(), 0.95)
            assert np.array_equal(view(momentum, i).cpu().numpy(), m)
            u = OM.muon_direction(m, view(grad, i).cpu().numpy(), 0.95, True)
            move = lr * OM.update_scale("rms", specs[i].rows, specs[i].cols) * OM.orthogonalize(u)
            want = view(before, i).double().cpu().numpy() * (1 - lr * 0.1) - move
            got = view(param, i).double().cpu().numpy()
            # sqrt(15) fp16 roundings of 2^-11 in the update, three fp32 ones beside it
            assert np.linalg.norm(got - want) <= 15 ** 0.5 * 2.0 ** -11 * np.linalg.norm(move) + 2.0 ** -22 * np.linalg.norm(want)
        # the rest moved by AdamW, bit for bit as the oracle's step, and has no momentum
        adam = OA.adam8_step(before.cpu().numpy(), grad.cpu().numpy(), *state, specs, starts, hyper)[0]
        for i in (0, 3):
            n_i = specs[i].rows * specs[i].cols
            assert np.array_equal(view(param, i).cpu().numpy().reshape(-1).view(np.uint32),
                                  np.asarray(adam)[starts[i]:starts[i] + n_i].view(np.uint32))
            assert not view(momentum, i).any()
        # steps that stay finite whatever AdamW did to the small values
        param.nan_to_num_(0.0).clamp_(-2.0, 2.0)
    plan.close()


def test_the_readme_example_of_these_calls_runs(gpu_lib):
    import structure_aware_grouped_amd as rs
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    block = re.search(r"same flat buffers \(imports as above\):\n\n((?:    .*\n|\n)+)", text).group(1)
    env = {"torch": torch, "rs": rs, "TensorSpec": TensorSpec}
    exec(compile(textwrap.dedent(block), "README.md", "exec"), env)
    torch.cuda.synchronize()
    (t, w), S = env["starts"], env["S"]
    table = env["gathered"][t:t + 32000 * 4096].view(32000, 4096)
    assert torch.equal(env["x"], table[env["ids"]] * 64)      # a power of two
    want = torch.zeros(32000, 4096, device=DEV).index_add_(0, env["ids"], env["x"].float())
    count = torch.zeros(32000, device=DEV).index_add_(0, env["ids"], torch.ones(2048, device=DEV))
    got = env["packed"][t:t + 32000 * 4096].view(32000, 4096) / 64
    # equal tokens have equal rows here: k - 1 roundings on either side of a sum of one sign
    assert bool(((got - want).abs() <= 2 * count[:, None] * 2.0 ** -24 * want.abs()).all())
    inside = torch.zeros(8 * S, dtype=torch.bool, device=DEV)
    inside[w:w + 4096 * 4096] = True
    assert torch.equal(env["momentum"], torch.where(inside, env["grads"], 0.0))   # 0.95 * 0 + g
    assert bool(torch.isfinite(env["params"]).all())
