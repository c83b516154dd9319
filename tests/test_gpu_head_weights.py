"""Tokens of weight 0 and tokens without a target add nothing to the head's
gradients, whatever finite values their x holds: x of all tokens is scaled to
fp16 by one power of two, which must be that of the tokens that count. Results
are compared bit for bit with those of a call whose masked tokens hold ordinary
values."""
import pytest
import torch

from tests.test_gpu_head import DT, Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("top", [0, 6])
@pytest.mark.parametrize("packed_dt", ["f32", "bf16"])
@pytest.mark.parametrize("piece", [0, 256])
@pytest.mark.parametrize("value", [2.0 ** 100, -1e30, 3.0e38, 2.0 ** 20])
def test_large_values_in_tokens_of_weight_zero(gpu_lib, top, packed_dt, piece, value):
    import structure_aware_grouped_amd as rs
    n, rows, cols = 300, 257, 72
    case = Case(rs, n, rows, cols, top=top, none=0.2)
    masked = torch.zeros(n, dtype=torch.bool, device=DEV)
    masked[[0, 17, 100, 299]] = True
    case.weights[masked] = 0.0
    case.weights[0] = -0.0
    outs = []
    for x in (case.x.clone(), case.x.clone()):
        if outs:
            x[masked] = value
        case.x = x
        packed = torch.zeros(case.total, device=DEV, dtype=DT[packed_dt])
        loss, dx = torch.zeros(n, device=DEV), torch.zeros(n, cols, device=DEV, dtype=torch.bfloat16)
        case.grad(rs, loss, dx, packed, case.work(rs, packed, piece), weights=case.weights, piece=piece)
        outs.append((loss, dx, packed))
    (loss, dx, packed), other = outs
    assert torch.equal(loss[~masked], other[0][~masked])
    assert torch.equal(dx, other[1]) and not bool(dx[masked].any())
    assert torch.equal(packed, other[2]) and bool(packed[case.at].any())
    case.plan.close()


@pytest.mark.parametrize("top", [0, 6])
def test_x_of_tokens_without_a_target_is_not_read(gpu_lib, top):
    """Whatever they hold, a call leaves the same bytes in a workspace that was cleared ahead of it."""
    import structure_aware_grouped_amd as rs
    n, rows, cols = 300, 257, 72
    case = Case(rs, n, rows, cols, top=top, none=0.4)
    live = torch.from_numpy(case.expect()["live"]).to(DEV)
    assert 0 < int(live.sum()) < n
    outs = []
    for value in (0.0, 2.0 ** 99, float("nan")):
        case.x[~live] = value
        packed = torch.zeros(case.total, device=DEV)
        loss, dx = torch.zeros(n, device=DEV), torch.zeros(n, cols, device=DEV, dtype=torch.bfloat16)
        work = case.work(rs, packed).zero_()
        case.grad(rs, loss, dx, packed, work)
        assert not bool(loss[~live].any()) and not bool(dx[~live].any())
        outs.append((work, loss, dx, packed))
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
    case.plan.close()


def test_temperatures_out_of_range_are_refused(gpu_lib):
    """A temperature whose square is 0 in fp32, and gradients whose common factor temperature * scale is not finite."""
    import structure_aware_grouped_amd as rs
    n = 10
    case = Case(rs, n, 100, 64, top=4)
    packed, loss, dx = torch.full((case.total,), 3.0, device=DEV), torch.full((n,), 3.0, device=DEV), torch.full_like(case.x, 3.0)
    work = case.work(rs, packed)
    args = (case.plan, 1, case.gathered, case.x, case.ids, case.teacher)
    for kw in ({"temperature": 1e-23}, {"temperature": 2.0 ** -76, "scale": 2.0 ** -20}):
        with pytest.raises(rs.RsError):
            rs.rs_distill_loss(*args, loss, work, **kw)
        with pytest.raises(rs.RsError):
            rs.rs_distill_grad(*args, loss, dx, packed, work, **kw)
    with pytest.raises(rs.RsError):
        rs.rs_distill_grad(*args, loss, dx, packed, work, temperature=1e18, scale=1e30)
    assert bool((packed == 3).all()) and bool((loss == 3).all()) and bool((dx == 3).all())
    case.plan.close()
