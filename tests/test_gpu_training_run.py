"""Several training steps one after the other on a plan's flat buffers, with
nothing between the calls that would hide a bad value: lookup, a small network
in torch, packed gradients with the tied table's added in place, the Muon step
on the matrices and the 8-bit AdamW step on the rest. AdamW's eps is a hundredth
of the gradients' size or more, so that a second moment whose code is zero
moves no parameter by more than its rate allows, and every step is checked
against the oracles from the state that the calls themselves left behind."""
import numpy as np
import pytest
import torch

from oracle import adam as OA, muon as OM
from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("parts", [1, 2])
def test_eight_steps_stay_finite_and_right(gpu_lib, parts):
    import structure_aware_grouped_amd as rs
    torch.manual_seed(4)
    vocab, d, h, n, V, lr, steps = 257, 96, 160, 220, 4, 0.02, 8
    specs = [TensorSpec("table", vocab, d, "TILE", 32, 32), TensorSpec("w1", h, d, "WHOLE"), TensorSpec("w2", d, h, "WHOLE"),
             TensorSpec("norm", d, 1, "FLAT", 64)]
    S, starts, _, _ = rs.rs_plan_build(specs, V)
    plan = rs.rs_plan_load(specs, V, S, starts, muon_parts=parts)
    total = V * S
    inside = torch.zeros(total, dtype=torch.bool, device=DEV)
    for sp, at in zip(specs, starts):
        inside[at:at + sp.rows * sp.cols] = True

    def view(flat, i):
        return flat[starts[i]:starts[i] + specs[i].rows * specs[i].cols].view(specs[i].rows, specs[i].cols)

    param = torch.zeros(total, device=DEV)
    for i, scale in enumerate((0.3, 0.1, 0.1, 1.0)):
        view(param, i).copy_(torch.randn(specs[i].rows, specs[i].cols, device=DEV) * scale)
    momentum, packed = torch.zeros(total, device=DEV), torch.zeros(total, device=DEV)
    codes = [torch.zeros(total, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.ones(plan.n_qblocks, device=DEV) for _ in range(2)]
    work, mwork = rs.rs_embed_workspace(plan, 0, n), rs.rs_muon_workspace(plan)
    ids, target = torch.randint(-1, vocab, (n,), device=DEV), torch.randint(0, vocab, (n,), device=DEV)
    adam = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-2, wd=0.01)
    largest, gmax = param.abs().max().item(), 0.0

    for step in range(1, steps + 1):
        gathered = param.clone()
        x = torch.empty(n, d, device=DEV)
        rs.rs_embed_rows(plan, 0, gathered, ids, x, scale=2.0)
        named = ids >= 0
        assert torch.equal(x, torch.where(named[:, None], view(gathered, 0)[ids.clamp(min=0)] * 2.0, 0.0))
        leaves = [view(gathered, i).clone().requires_grad_() for i in range(4)]
        xin = x.clone().requires_grad_()
        y = torch.nn.functional.silu(xin @ leaves[1].T) @ leaves[2].T
        y = (xin + y) * leaves[3].view(1, d)
        torch.nn.functional.cross_entropy(y @ leaves[0].T, target).backward()
        rs.rs_pack_scatter(plan, [l.grad.contiguous() for l in leaves], packed)
        dense = view(packed, 0).double().clone()
        rs.rs_embed_grad(plan, 0, ids, xin.grad, packed, work, prev=packed, scale=2.0, inv_v=True)
        more = torch.zeros(vocab, d, dtype=torch.float64, device=DEV).index_add_(0, ids[named], xin.grad[named].double()) * (2.0 / V)
        size = torch.zeros(vocab, d, dtype=torch.float64, device=DEV).index_add_(0, ids[named], xin.grad[named].abs().double()) * (2.0 / V)
        # up to n additions, one product and one addition to the dense gradient, 2^-24 each
        assert bool(((view(packed, 0).double() - dense - more).abs() <= 2.0 ** -24 * ((n + 1) * size + (dense + more).abs()) * 1.001).all())
        assert bool(torch.isfinite(packed).all()) and not packed[~inside].any()

        before, mom_before, grad = param.clone(), momentum.clone(), packed.clone()
        rs.rs_muon_step(plan, param, packed, momentum, mwork, lr=lr, weight_decay=0.1, update_scale="spectral")
        state = [t.cpu().numpy().copy() for t in (codes[0], scales[0], codes[1], scales[1])]
        hyper = OA.AdamHyper(adam["lr"], adam["beta1"], adam["beta2"], adam["eps"], adam["wd"], step)
        rs.rs_adam8_step(plan, param, packed, codes[0], scales[0], codes[1], scales[1], adam["lr"], adam["beta1"],
                         adam["beta2"], adam["eps"], adam["wd"], step)
        torch.cuda.synchronize()
        for i in (1, 2):
            m = OM.momentum_f32(view(mom_before, i).cpu().numpy(), view(grad, i).cpu().numpy(), 0.95)
            assert np.array_equal(view(momentum, i).cpu().numpy(), m)
            move = lr * OM.update_scale("spectral", specs[i].rows, specs[i].cols) * OM.orthogonalize(
                OM.muon_direction(m, view(grad, i).cpu().numpy(), 0.95, True))
            want = view(before, i).double().cpu().numpy() * (1 - lr * 0.1) - move
            got = view(param, i).double().cpu().numpy()
            # sqrt(15) fp16 roundings of 2^-11 in the update (no more with two parts), three fp32 ones beside it
            assert np.linalg.norm(got - want) <= 15 ** 0.5 * 2.0 ** -11 * np.linalg.norm(move) + 2.0 ** -22 * np.linalg.norm(want)
        want = OA.adam8_step(before.cpu().numpy(), grad.cpu().numpy(), *state, specs, starts, hyper)[0]
        for i in (0, 3):
            n_i = specs[i].rows * specs[i].cols
            assert np.array_equal(view(param, i).cpu().numpy().reshape(-1).view(np.uint32),
                                  np.asarray(want)[starts[i]:starts[i] + n_i].view(np.uint32))
            assert not view(momentum, i).any()
        # no value is replaced, and none runs away: AdamW moves one by at most its rate times |m| / eps, with |m| below
        # twice the largest gradient so far (codes of m round by 1/254 of a block's largest a step), Muon's update has
        # singular values of at most 1.3 times lr * sqrt(160 / 96), and both decay
        assert bool(torch.isfinite(param).all()) and not param[~inside].any() and not momentum[~inside].any()
        gmax = max(gmax, grad.abs().max().item())
        moved = (param - before).abs().max().item()
        assert moved <= max(adam["lr"] / adam["eps"] * 2 * gmax, 1.3 * lr * (160 / 96) ** 0.5) + 0.1 * lr * largest
        largest = param.abs().max().item()
        ids = torch.randint(-1, vocab, (n,), device=DEV)
        target = torch.randint(0, vocab, (n,), device=DEV)
    plan.close()
