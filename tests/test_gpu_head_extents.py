"""The head's calls at the ends of their ranges: tables and logits past 2^32
bytes and 2^31 elements, a workspace meant for more tokens, ids at any multiple
of their size, calls on another stream than the current one.

References are products of the same bf16 values in 64 bits on the device, a few
tokens or rows at a time. Tolerances as in test_gpu_head.py: an fp32 sum of k
products is off by at most 2 k 2^-24 of the sum of absolute values, d by its
rounding (2^-8 for dx, 2^-22 for an fp32 table)."""
import pytest
import torch

from tests.test_gpu_head import Case, _check_grad, _f64
from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def _load(rs, rows, cols):
    specs = [TensorSpec("head", rows, cols, "ROWS", 1)]
    S, starts, _, _ = rs.rs_plan_build(specs, 1)
    return rs.rs_plan_load(specs, 1, S, starts, 1, 0)


def test_logits_past_2_to_32_bytes(gpu_lib):
    """2^21 - 3 rows, 1100 tokens in one piece: 2.3e9 logits, 9.2e9 bytes, in blocks past 2^31 elements."""
    import structure_aware_grouped_amd as rs
    rows, cols, n = (1 << 21) - 3, 16, 1100
    plan = _load(rs, rows, cols)
    gen = torch.Generator(device=DEV).manual_seed(3)
    flat = torch.zeros(plan.S, dtype=torch.bfloat16, device=DEV)
    table = flat[:rows * cols].view(rows, cols)
    table.copy_(torch.randn(rows, cols, device=DEV, generator=gen))
    x = torch.randn(n, cols, device=DEV, generator=gen).to(torch.bfloat16)
    y = torch.randint(rows - 5000, rows, (n,), device=DEV, generator=gen)
    y[::2] = torch.randint(0, 5000, (n // 2,), device=DEV, generator=gen)
    weights = torch.rand(n, device=DEV, generator=gen)
    loss, dx = torch.empty(n, device=DEV), torch.empty_like(x)
    packed = torch.full((plan.S,), float("nan"), device=DEV)
    work = rs.rs_head_workspace(plan, 0, n, packed=packed)
    assert work.numel() > 2 ** 32
    rs.rs_head_grad(plan, 0, flat, x, y, loss, dx, packed, work, weights=weights, scale=0.5)
    w64 = table.double()
    for t0 in (0, 512, 1036):
        t = slice(t0, t0 + 64)
        l = 0.5 * x[t].double() @ w64.T
        z = l.logsumexp(1)
        at = torch.arange(64, device=DEV)
        # logits: 2 (16 + 2) u of 0.5 sum |x w| <= 120; the log-sum: 1134 u and an exponent's 4 u + |l - z| u
        assert float((loss[t].double() - (z - l[at, y[t]])).abs().max()) <= 36 * U * 120 + 1300 * U
        p = (l - z[:, None]).exp_()
        p[at, y[t]] -= 1.0
        want = 0.5 * weights[t].double()[:, None] * (p @ w64)
        absolute = 0.5 * weights[t].double()[:, None] * (p.abs() @ w64.abs())
        # d: its rounding 2^-8 and the logits' errors 6e-4; parts of the sum are joined, chains of at most 8192 rows
        off = absolute * (2.0 ** -8 + 2e-3 + 2 * 9000 * U) + 2.0 ** -8 * want.abs()
        assert bool(((dx[t].double() - want).abs() <= off).all())
    lse = torch.cat([(0.5 * x[t:t + 64].double() @ w64.T).logsumexp(1) for t in range(0, n, 64)])
    got = packed[:rows * cols].view(rows, cols)
    for r0 in (0, 4096, rows // 2, rows - 4096):
        d = (0.5 * x.double() @ w64[r0:r0 + 4096].T - lse[:, None]).exp_()
        own = ((y >= r0) & (y < r0 + 4096)).nonzero().ravel()
        d[own, y[own] - r0] -= 1.0
        d *= 0.5 * weights.double()[:, None]
        want, absolute = d.T @ x.double(), d.abs().T @ x.double().abs()
        off = absolute * (2.0 ** -22 + 1e-3 + 2 * n * U) + 2.0 ** -38 * x.double().abs().sum(0)
        assert bool(((got[r0:r0 + 4096].double() - want).abs() <= off).all())
    assert bool(torch.isfinite(got).all())
    plan.close()


def test_a_table_of_more_than_2_to_31_elements(gpu_lib):
    """Rows on both sides of element 2^31 (byte 2^32 of the gathered buffer, 2^33 of the packed one)."""
    import structure_aware_grouped_amd as rs
    rows, cols, n = 36000, 60000, 5                        # 2.16e9 elements; 2^31 lies in row 35791
    plan = _load(rs, rows, cols)
    gen = torch.Generator(device=DEV).manual_seed(4)
    flat = torch.zeros(plan.S, dtype=torch.bfloat16, device=DEV)
    table = flat[:rows * cols].view(rows, cols)
    mark = torch.tensor([0, 17895, 35790, 35791, 35792, rows - 1], device=DEV)
    table[mark] = (torch.randn(mark.numel(), cols, device=DEV, generator=gen) * 2.0 ** -6).to(torch.bfloat16)
    x = torch.randn(n, cols, device=DEV, generator=gen).to(torch.bfloat16)
    y = torch.tensor([0, 35790, 35791, rows - 1, -1], device=DEV)
    loss, dx = torch.empty(n, device=DEV), torch.empty_like(x)
    packed = torch.full((plan.S,), float("nan"), device=DEV)
    rs.rs_head_grad(plan, 0, flat, x, y, loss, dx, packed, rs.rs_head_workspace(plan, 0, n, packed=packed))
    x64, w64 = x[:4].double(), table[mark].double()
    l = x64 @ w64.T                                        # the other rows' logits are 0
    z = torch.cat([l, torch.zeros(4, 1, device=DEV, dtype=torch.float64)], 1)
    z[:, -1] = torch.log(torch.tensor(float(rows - mark.numel()), dtype=torch.float64))
    z = z.logsumexp(1)
    hit = y[:4, None] == mark[None]
    # logits: 60000 / 16 additions in the matrix cores, each off by at most two half steps of a partial sum, and
    # partial sums of random signs (deviation 2^-6 sqrt(60000) = 3.9) stay under 40
    off_l = 2 * 3752 * U * 40
    assert float((loss[:4].double() - (z - (l * hit).sum(1))).abs().max()) <= 2 * off_l + 200 * U and float(loss[4]) == 0.0
    d = (l - z[:, None]).exp() - hit.double()
    want, absolute = d @ w64, d.abs() @ w64.abs()
    off = absolute * (2.0 ** -8 + 4 * off_l + 2 * rows * U) + 2.0 ** -8 * want.abs()
    assert bool(((dx[:4].double() - want).abs() <= off).all()) and not bool(dx[4].any())
    got = packed[:rows * cols].view(rows, cols)
    want, absolute = d.T @ x64, d.abs().T @ x64.abs()
    off = absolute * (2.0 ** -22 + 4 * off_l + 20 * U) + 2.0 ** -38 * x64.abs().sum(0)
    for i, r in enumerate(mark.tolist()):
        assert bool(((got[r].double() - want[i]).abs() <= off[i]).all()), r
    rest = (0.0 - z).exp() @ x64                           # every other row: p alone
    off = (0.0 - z).exp() @ x64.abs() * (2.0 ** -22 + 4 * off_l + 20 * U) + 2.0 ** -38 * x64.abs().sum(0)
    for r in (1, 17894, 17896, 35789, 35793, rows - 2):
        assert bool(((got[r].double() - rest).abs() <= off).all()), r
    plan.close()


@pytest.mark.parametrize("top", [0, 9])
def test_a_workspace_for_more_tokens(gpu_lib, top):
    """One workspace for the largest batch, gradients and losses, batches of fewer tokens in any order."""
    import structure_aware_grouped_amd as rs
    big = Case(rs, 600, 900, 72, top=top)
    packed = torch.zeros(big.total, device=DEV)
    work = rs.rs_head_workspace(big.plan, 1, 600, top=top, packed=packed, piece=256)
    for n in (600, 64, 257, 1, 128, 512, 65):
        case = Case(rs, n, 900, 72, top=top, seed=n)
        case.work = lambda rs, packed=None, piece=0: work      # with what the last call left in it
        _check_grad(rs, case, "f32", piece=256)
        loss = torch.empty(n, device=DEV)
        case.loss(rs, loss, work, piece=256)
        want = case.expect()
        assert (abs(_f64(loss) - want["loss"]) <= want["off_loss"]).all()
        case.plan.close()
    big.plan.close()


@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
def test_targets_at_any_multiple_of_their_size(gpu_lib, idx):
    import structure_aware_grouped_amd as rs
    for top in (0, 3):
        case = Case(rs, 70, 300, 40, top=top, idx=idx)
        room = torch.empty(case.ids.numel() + 1, dtype=idx, device=DEV)
        room[1:] = case.ids.ravel()
        case.ids = room[1:].view(case.ids.shape)
        _check_grad(rs, case, "bf16")
        case.plan.close()


def test_another_stream_than_the_current_one(gpu_lib):
    """The call goes to the stream that is current when it is made, in order with that stream's own work."""
    import structure_aware_grouped_amd as rs
    case = Case(rs, 300, 1025, 65)
    want = case.expect()
    side, loss = torch.cuda.Stream(), torch.zeros(300, device=DEV)
    work, x = case.work(rs), case.x.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        case.x.zero_()
        torch.cuda._sleep(2_000_000)
        case.x.copy_(x)
        case.loss(rs, loss, work)
        after = loss.clone()
    side.synchronize()
    assert (abs(_f64(after) - want["loss"]) <= want["off_loss"]).all()
    case.plan.close()


def test_both_parts_of_d_are_of_one_value(gpu_lib):
    """fp32 gradients of a table keep 22 bits of d in every one of 200000 rows, also where a value lies halfway
    between two of its first part.

    x and the table are small: the logits are off by 2 (64 + 2) u sum |x w| <= 132 u, the log-sum by that and
    64 + 1 + 200000 / 2048 + 32 + 8 = 203 u, the exponential by 4 u and the result by two steps more: 480 u and
    the parts' 2^-22, under 2^-15. A first part a step away would be off by 2^-11 to 2^-10."""
    import structure_aware_grouped_amd as rs
    rows, cols = 200000, 64
    plan = _load(rs, rows, cols)
    gen = torch.Generator(device=DEV).manual_seed(6)
    flat = torch.zeros(plan.S, dtype=torch.bfloat16, device=DEV)
    table = flat[:rows * cols].view(rows, cols)
    table.copy_(torch.rand(rows, cols, device=DEV, generator=gen) * 2 - 1)
    x = ((torch.rand(1, cols, device=DEV, generator=gen) + 0.5) * 2.0 ** -7).to(torch.bfloat16)
    y, weights = torch.tensor([7], device=DEV), torch.tensor([0.7361], device=DEV)
    loss, dx, packed = torch.empty(1, device=DEV), torch.empty_like(x), torch.empty(plan.S, device=DEV)
    rs.rs_head_grad(plan, 0, flat, x, y, loss, dx, packed, rs.rs_head_workspace(plan, 0, 1, packed=packed), weights=weights)
    l = table.double() @ x[0].double()
    assert float((table.double().abs() @ x[0].double().abs()).max()) <= 1.0
    d = (l - l.logsumexp(0)).exp()
    d[7] -= 1.0
    want = weights[0].double() * d[:, None] * x.double()
    got = packed[:rows * cols].view(rows, cols).double()
    assert bool(((got - want).abs() <= 2.0 ** -15 * want.abs()).all())
    plan.close()


@pytest.mark.parametrize("n,rows,cols,top", [(300, 700, 2049, 0), (257, 300, 2112, 0), (300, 520, 2304, 7), (1, 300, 2112, 0), (70, 300, 2100, 3)])
def test_long_rows(gpu_lib, n, rows, cols, top):
    import structure_aware_grouped_amd as rs
    case = Case(rs, n, rows, cols, top=top)
    want = case.expect()
    loss = torch.full((n,), float("nan"), device=DEV)
    case.loss(rs, loss, case.work(rs))
    assert (abs(_f64(loss) - want["loss"]) <= want["off_loss"]).all()
    _check_grad(rs, case, "f32")
    _check_grad(rs, case, "bf16", mode="other", inv_v=True)
    case.plan.close()
