"""rs_embed_rows and rs_embed_grad against the CPU oracle.

The lookup is one fp32 product and at most one rounding to bf16: bit for bit.
The gradient sums k fp32 values in some fixed order: at most (k - 1) additions
of at most 2^-24 each relative to the sum of the absolute values, one more
rounding for the scale and one for prev, and half a bf16 step (2^-8 of the
value) where the buffer is bf16. Sums of small whole numbers are exact."""
import numpy as np
import pytest
import torch

from oracle import embed as OE
from tests.gpu_util import guard_intact, guarded, tensor_bits
from workloads import TensorSpec, bf16_bits_from_f32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _load(rs, specs, V):
    S, starts, _, _ = rs.rs_plan_build(specs, V)
    return rs.rs_plan_load(specs, V, S, starts, V, 0)


def _group(rs, rows, cols, kind=("ROWS", 1, 0), V=3):
    """A table between two other tensors."""
    return _load(rs, [TensorSpec("before", 37, 5, "ELEM"), TensorSpec("table", rows, cols, *kind),
                      TensorSpec("after", 20, 20, "WHOLE")], V)


def _ids(rng, n, rows, kind):
    if kind == "same":
        return np.full(n, rows // 2)
    if kind == "few":
        ids = rng.choice(rng.integers(0, rows, 3), n)
    elif kind == "power":
        ids = np.minimum(rows - 1, np.floor(rows ** rng.random(n) - 1).astype(np.int64))
    else:
        ids = rng.integers(0, rows, n)
    ids = ids.copy()
    if kind == "padded":                    # ids that name no row, at both ends of the range
        bad = rng.random(n) < 0.4
        ids[bad] = rng.choice([-1, -7, rows, rows + 3, 2 ** 31 - 1, -2 ** 31], bad.sum())
    if kind == "none":
        ids[:] = -1
    return ids


def _bits(x, dt):
    return x.view(np.uint32) if dt == "f32" else bf16_bits_from_f32(x)


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 7), (50, 8), (300, 64), (129, 1001), (1000, 2880), (64, 8200)])
@pytest.mark.parametrize("dt,out_dt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_lookup_bit_for_bit(gpu_lib, rows, cols, dt, out_dt):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(rows * 31 + cols)
    plan = _group(rs, rows, cols)
    at = plan.starts[1]
    flat = torch.full((plan.R_mat * plan.S,), float("nan"), dtype=DT[dt], device=DEV)
    flat[at:at + rows * cols] = torch.randn(rows * cols, device=DEV).to(DT[dt])
    table = flat[at:at + rows * cols].float().cpu().numpy().reshape(rows, cols)
    for n in (0, 1, 3, 64, 257, 1000):
        for kind in ("uniform", "padded"):
            for it in (torch.int32, torch.int64):
                ids = _ids(rng, n, rows, kind)
                scale = float(rng.choice([1.0, 64.0, -0.37, 0.0]))
                whole, out = guarded(n * cols, DT[out_dt], DEV)
                rs.rs_embed_rows(plan, 1, flat, torch.from_numpy(ids).to(it).to(DEV), out, scale=scale)
                torch.cuda.synchronize()
                want = _bits(OE.lookup(table, ids, scale).reshape(-1), out_dt)
                assert np.array_equal(tensor_bits(out), want), (n, kind, it, scale)
                assert guard_intact(whole, n * cols)
    plan.close()


def test_large_int64_ids_name_no_row(gpu_lib):
    import structure_aware_grouped_amd as rs
    plan = _group(rs, 10, 8)
    flat = torch.ones(plan.R_mat * plan.S, device=DEV)
    ids = torch.tensor([2 ** 32, 2 ** 32 + 3, -2 ** 63, 2 ** 63 - 1, 3], device=DEV)
    out = torch.full((5, 8), 9.0, device=DEV)
    rs.rs_embed_rows(plan, 1, flat, ids, out)
    assert out.sum(1).tolist() == [0, 0, 0, 0, 8]
    packed = torch.zeros_like(flat)
    rs.rs_embed_grad(plan, 1, ids, torch.ones(5, 8, device=DEV), packed, rs.rs_embed_workspace(plan, 1, 5))
    assert packed.sum().item() == 8 and packed[plan.starts[1] + 24].item() == 1
    plan.close()


@pytest.mark.parametrize("kind", [("ELEM", 0, 0), ("ROWS", 7, 0), ("TILE", 16, 16), ("FLAT", 100, 0), ("WHOLE", 0, 0)])
def test_every_row_major_block_kind(gpu_lib, kind):
    import structure_aware_grouped_amd as rs
    plan = _group(rs, 60, 24, kind, V=4)
    flat = torch.randn(plan.R_mat * plan.S, device=DEV)
    ids = torch.randint(0, 60, (50,), device=DEV)
    out = torch.empty(50, 24, device=DEV)
    rs.rs_embed_rows(plan, 1, flat, ids, out)
    at = plan.starts[1]
    assert torch.equal(out, flat[at:at + 60 * 24].view(60, 24)[ids])
    plan.close()


def _grad_case(rs, plan, rows, cols, ids, it, dt, packed_dt, mode, scale, inv_v, dy):
    at, total = plan.starts[1], plan.R_mat * plan.S
    d = torch.from_numpy(dy).to(DEV).to(DT[dt])
    work = rs.rs_embed_workspace(plan, 1, ids.size)
    work.fill_(0xFF)
    rng = np.random.default_rng(1)
    base = rng.integers(-50, 50, total).astype(np.float32)
    packed = torch.from_numpy(base).to(DEV).to(DT[packed_dt])
    before = packed.clone()
    prev = None
    if mode == "add":
        prev = packed
    elif mode == "prev":
        base = rng.integers(-50, 50, total).astype(np.float32)
        prev = torch.from_numpy(base).to(DEV)
    rs.rs_embed_grad(plan, 1, torch.from_numpy(ids).to(it).to(DEV), d, packed, work, prev=prev, scale=scale, inv_v=inv_v)
    torch.cuda.synchronize()
    outside = torch.ones(total, dtype=torch.bool, device=DEV)
    outside[at:at + rows * cols] = False
    assert torch.equal(packed[outside], before[outside])
    got = packed[at:at + rows * cols].double().cpu().numpy().reshape(rows, cols)
    s, size, count = OE.row_sums(d.double().cpu().numpy(), ids, rows)
    sg = np.float64(OE.sigma(scale, inv_v, plan.V))
    want, err = s * sg, (size * count[:, None] + np.abs(s)) * abs(sg) * 2.0 ** -24
    if mode != "write":
        want = want + base[at:at + rows * cols].reshape(rows, cols)
        err = err + np.abs(want) * 2.0 ** -24
    if packed_dt == "bf16":
        err = err * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8
    return got, want, err * (1 + 2.0 ** -20)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (40, 8), (129, 1001), (500, 260), (70, 4100)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("mode,packed_dt", [("write", "f32"), ("write", "bf16"), ("add", "f32"), ("prev", "f32"), ("prev", "bf16")])
def test_gradient_matches_64_bits(gpu_lib, rows, cols, dt, mode, packed_dt):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(rows * 77 + cols)
    plan = _group(rs, rows, cols)
    for n in (0, 1, 2, 63, 64, 65, 500, 2048, 2049) if cols < 1000 else (1, 130, 700):
        for kind in ("uniform", "power", "same", "few", "padded", "none"):
            ids = _ids(rng, n, rows, kind)
            it = torch.int64 if rng.random() < 0.5 else torch.int32
            scale, inv_v = [(1.0, False), (0.125, True), (31.6, False)][rng.integers(3)]
            dy = rng.standard_normal((n, cols)).astype(np.float32)
            got, want, err = _grad_case(rs, plan, rows, cols, ids, it, dt, packed_dt, mode, scale, inv_v, dy)
            assert (np.abs(got - want) <= err).all(), (n, kind, float((np.abs(got - want) - err).max()))
    plan.close()


def test_sums_of_whole_numbers_are_exact_over_many_runs(gpu_lib):
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(5)
    rows, cols, n = 3000, 12, 40_003            # 20 sorted runs, the last one partial
    plan = _group(rs, rows, cols)
    for kind in ("uniform", "power", "few", "padded"):
        ids = _ids(rng, n, rows, kind)
        dy = rng.integers(-8, 9, (n, cols)).astype(np.float32)
        for mode in ("write", "add"):
            got, want, _ = _grad_case(rs, plan, rows, cols, ids, torch.int64, "f32", "f32", mode, 1.0, False, dy)
            assert np.array_equal(got, want), (kind, mode)
    plan.close()


@pytest.mark.parametrize("packed_dt,with_prev", [("f32", False), ("f32", True), ("bf16", False), ("bf16", True)])
def test_a_large_table_is_filled_to_both_ends(gpu_lib, packed_dt, with_prev):
    """More rows without a token than the sort's launch fills (96 MiB): the rest is the chunk sums'
    launch's. Whole numbers: sums, prev and the bf16 results (below 256) are exact."""
    import structure_aware_grouped_amd as rs
    rows, cols, n = 12007, 4501, 300
    plan = _group(rs, rows, cols)
    at, total = plan.starts[1], plan.R_mat * plan.S
    ids = torch.randint(0, 40, (n,), device=DEV) * 300
    ids[:2] = torch.tensor([0, rows - 1], device=DEV)
    dy = torch.randint(-1, 2, (n, cols), device=DEV).float()
    packed = torch.full((total,), float("nan"), dtype=DT[packed_dt], device=DEV)
    prev = torch.randint(-3, 4, (total,), device=DEV).float() if with_prev else None
    rs.rs_embed_grad(plan, 1, ids, dy, packed, rs.rs_embed_workspace(plan, 1, n), prev=prev)
    want = torch.zeros(rows, cols, device=DEV) if prev is None else prev[at:at + rows * cols].view(rows, cols).clone()
    want.index_add_(0, ids, dy)
    assert want.abs().max().item() < 256
    assert torch.equal(packed[at:at + rows * cols].float().view(rows, cols), want)
    assert bool(torch.isnan(packed[:at]).all()) and bool(torch.isnan(packed[at + rows * cols:]).all())
    plan.close()


def test_same_call_same_bits_and_no_read_of_padding_tokens(gpu_lib):
    import structure_aware_grouped_amd as rs
    plan = _group(rs, 200, 100)
    n = 6000
    ids = torch.randint(0, 20, (n,), device=DEV)
    ids[::3] = -1
    dy = torch.randn(n, 100, device=DEV)
    dy[::3] = float("nan")
    work = rs.rs_embed_workspace(plan, 1, n)
    a, b = torch.zeros(plan.R_mat * plan.S, device=DEV), torch.zeros(plan.R_mat * plan.S, device=DEV)
    rs.rs_embed_grad(plan, 1, ids, dy, a, work)
    rs.rs_embed_grad(plan, 1, ids, dy, b, work)
    assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    plan.close()


def test_gradient_agrees_with_differences_of_the_lookup(gpu_lib):
    """sum(w * lookup(table)) is linear in the table: its difference along any direction is the
    gradient's product with that direction."""
    import structure_aware_grouped_amd as rs
    rng = np.random.default_rng(6)
    rows, cols, n, scale = 30, 20, 90, 4.0
    plan = _group(rs, rows, cols)
    total = plan.R_mat * plan.S
    flat = torch.from_numpy(rng.integers(-4, 5, total).astype(np.float32)).to(DEV)
    ids = torch.from_numpy(_ids(rng, n, rows, "padded")).to(DEV)
    w = torch.from_numpy(rng.integers(-4, 5, (n, cols)).astype(np.float32)).to(DEV)
    packed = torch.zeros(total, device=DEV)
    rs.rs_embed_grad(plan, 1, ids, w, packed, rs.rs_embed_workspace(plan, 1, n), scale=scale)
    lo, hi = torch.empty(n, cols, device=DEV), torch.empty(n, cols, device=DEV)
    for _ in range(5):                          # whole numbers: every product and sum is exact
        step = torch.from_numpy(rng.integers(-3, 4, total).astype(np.float32)).to(DEV)
        rs.rs_embed_rows(plan, 1, flat, ids, lo, scale=scale)
        rs.rs_embed_rows(plan, 1, flat + step, ids, hi, scale=scale)
        assert ((hi - lo) * w).double().sum().item() == (packed * step).double().sum().item()
    plan.close()


def test_captured_lookup_and_gradient(gpu_lib):
    import structure_aware_grouped_amd as rs
    plan = _group(rs, 400, 96)
    total, n = plan.R_mat * plan.S, 5000
    flat, ids = torch.randn(total, device=DEV), torch.randint(0, 400, (n,), device=DEV)
    out, packed = torch.empty(n, 96, device=DEV), torch.zeros(total, device=DEV)
    work = rs.rs_embed_workspace(plan, 1, n)

    def step(o, p, w):
        rs.rs_embed_rows(plan, 1, flat, ids, o, scale=2.0)
        rs.rs_embed_grad(plan, 1, ids, o, p, w, prev=p)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, packed, work)
    ref_out, ref, ref_work = torch.empty_like(out), torch.zeros_like(packed), torch.empty_like(work)
    for _ in range(3):
        ids.copy_(torch.randint(-2, 400, (n,), device=DEV))
        torch.cuda.synchronize()
        graph.replay()
        step(ref_out, ref, ref_work)
        torch.cuda.synchronize()
        assert torch.equal(out, ref_out) and torch.equal(packed, ref)
    del graph
    plan.close()


def test_calls_that_are_refused(gpu_lib):
    import structure_aware_grouped_amd as rs
    from structure_aware_grouped_amd import binding as b
    specs = [TensorSpec("tm", 32, 32, "TILEMAJOR", 16, 16), TensorSpec("t", 32, 32, "ROWS", 1)]
    plan = _load(rs, specs, 2)
    flat = torch.zeros(plan.R_mat * plan.S, device=DEV)
    ids, dy = torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, 32, device=DEV)
    work = rs.rs_embed_workspace(plan, 1, 4)

    def status(fn):
        with pytest.raises(rs.RsError) as e:
            fn()
        return e.value.status

    assert status(lambda: rs.rs_embed_rows(plan, 0, flat, ids, dy)) == b.RS_EINVAL
    assert status(lambda: rs.rs_embed_workspace(plan, 0, 4)) == b.RS_EINVAL
    assert status(lambda: rs.rs_embed_workspace(plan, 2, 4)) == b.RS_EINVAL
    assert status(lambda: rs.rs_embed_workspace(plan, 1, -1)) == b.RS_EINVAL
    assert status(lambda: rs.rs_embed_workspace(plan, 1, 2 ** 26)) == b.RS_ERANGE
    assert status(lambda: rs.rs_embed_rows(plan, 1, flat, ids, dy, scale=float("inf"))) == b.RS_EINVAL
    assert status(lambda: rs.rs_embed_grad(plan, 1, ids, dy, flat, work, scale=float("nan"))) == b.RS_EINVAL
    lib, h = b.load(), plan.handle
    assert lib.rs_embed_rows(h, 1, flat.data_ptr(), 0, ids.data_ptr(), 2, 4, 1.0, dy.data_ptr(), 0, None) == b.RS_EINVAL
    assert lib.rs_embed_rows(h, 1, flat.data_ptr(), 0, ids.data_ptr() + 4, 8, 3, 1.0, dy.data_ptr(), 0, None) == b.RS_EALIGN
    assert lib.rs_embed_rows(h, 1, flat.data_ptr(), 2, ids.data_ptr(), 8, 4, 1.0, dy.data_ptr(), 0, None) == b.RS_EDTYPE
    assert lib.rs_embed_rows(h, 1, flat.data_ptr(), 0, None, 8, 4, 1.0, dy.data_ptr(), 0, None) == b.RS_EINVAL
    args = (h, 1, ids.data_ptr(), 8, 4, dy.data_ptr(), 0)
    wk = (work.data_ptr(), work.numel(), None)
    half = torch.zeros(flat.numel(), dtype=torch.bfloat16, device=DEV)
    assert lib.rs_embed_grad(*args, half.data_ptr(), half.data_ptr(), 1, 1, 1.0, *wk) == b.RS_EINVAL
    assert lib.rs_embed_grad(*args, None, flat.data_ptr(), 0, 2, 1.0, *wk) == b.RS_EINVAL
    assert lib.rs_embed_grad(*args, None, flat.data_ptr(), 0, 1, 1.0, work.data_ptr(), 0, None) == b.RS_EINVAL
    assert lib.rs_embed_grad(*args, None, flat.data_ptr(), 0, 1, 1.0, None, 0, None) == b.RS_EINVAL
    torch.cuda.synchronize()
    assert not flat.any() and not half.any()
    plan.close()
