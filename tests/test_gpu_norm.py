"""rs_layer_norm and rs_layer_norm_grad against the 64-bit oracle.

Tolerances. With u = 2^-24 (half an fp32 step): a sum over a row of at most
16384 values is a chain of at most 16 + 6 + 16 additions (values of a thread,
lanes, waves), so a row's sums are off by at most 40 u of the sum of absolute
values, and each step after them by u. With A = r mean|x| (what an error of the
mean costs, in units of the result) a value h is off by at most 64 u (|h| + A).
Weight gradients add rows in chains of at most n / 256 + 300. A bf16 result has
half a step more, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from oracle import norm as ON
from tests.gpu_util import guard_intact, guarded
from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = {"f32": 0.0, "bf16": 2.0 ** -8}
U = 2.0 ** -24
COLS = [1, 7, 8, 63, 64, 100, 513, 1001, 2048, 4096, 5000, 8192, 9001, 16384]


def _plan(rs, cols, V=3):
    specs = [TensorSpec("before", 37, 5, "ELEM"), TensorSpec("w", cols, 1, "ROWS", 1), TensorSpec("b", 1, cols, "WHOLE"),
             TensorSpec("tiles", 32, 32, "TILEMAJOR", 16, 16)]
    S, starts, _, _ = rs.rs_plan_build(specs, V)
    return rs.rs_plan_load(specs, V, S, starts, V, 0)


def _gathered(plan, dt, gen):
    """The parameters, NaN everywhere else."""
    flat = torch.full((plan.R_mat * plan.S,), float("nan"), device=DEV)
    for t, mean in ((1, 1.0), (2, 0.0)):
        n = plan.numels[t]
        flat[plan.starts[t]:plan.starts[t] + n] = mean + 0.5 * torch.randn(n, device=DEV, generator=gen)
    return flat.to(DT[dt])


def _param(plan, flat, t):
    return flat[plan.starts[t]:plan.starts[t] + plan.numels[t]].double().cpu().numpy()


def _f64(t):
    return t.double().cpu().numpy()


def _parts(x, eps, center):
    h, r = ON._parts(x, eps, center)
    return h, r, r * np.abs(x).mean(1, keepdims=True)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt,out_dt,param_dt", [("f32", "f32", "f32"), ("f32", "bf16", "bf16"), ("bf16", "f32", "bf16"),
                                                ("bf16", "bf16", "f32")])
def test_forward(gpu_lib, cols, dt, out_dt, param_dt):
    import structure_aware_grouped_amd as rs
    gen = torch.Generator(device=DEV).manual_seed(cols)
    plan = _plan(rs, cols)
    flat = _gathered(plan, param_dt, gen)
    w, b = _param(plan, flat, 1), _param(plan, flat, 2)
    for n in (0, 1, 2, 67):
        x = (torch.randn(n, cols, device=DEV, generator=gen) * 3 + 2).to(DT[dt])
        for center, bias in ((True, 2), (True, None), (False, None), (False, 2)):
            whole, y = guarded(n * cols, DT[out_dt], DEV)
            rs.rs_layer_norm(plan, 1, flat, x, y, bias=bias, eps=1e-5, center=center)
            assert guard_intact(whole, n * cols)
            if not n:
                continue
            xd = _f64(x)
            want = ON.norm(xd, w, b if bias else None, 1e-5, center)
            h, _, a = _parts(xd, 1e-5, center)
            off = 64 * U * (np.abs(h) + a) * np.abs(w) + 4 * U * np.abs(want) + 4 * U * (np.abs(b) if bias else 0.0)
            off += STEP[out_dt] * (np.abs(want) + off)
            assert (np.abs(_f64(y).reshape(n, cols) - want) <= off).all(), (n, center, bias)
    plan.close()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt,dy_dt,param_dt,packed_dt", [("f32", "f32", "f32", "f32"), ("f32", "bf16", "bf16", "bf16"),
                                                         ("bf16", "f32", "bf16", "f32"), ("bf16", "bf16", "f32", "bf16")])
def test_gradients(gpu_lib, cols, dt, dy_dt, param_dt, packed_dt):
    import structure_aware_grouped_amd as rs
    gen = torch.Generator(device=DEV).manual_seed(cols)
    plan = _plan(rs, cols)
    flat = _gathered(plan, param_dt, gen)
    w = _param(plan, flat, 1)
    total = plan.R_mat * plan.S
    for n in (0, 1, 3, 300, 2111):
        x = (torch.randn(n, cols, device=DEV, generator=gen) * 2 + 1).to(DT[dt])
        dy = torch.randn(n, cols, device=DEV, generator=gen).to(DT[dy_dt])
        work = rs.rs_layer_norm_workspace(plan, 1, n)
        modes = [(True, 2, "none"), (False, None, "prev")] + ([(True, None, "in place")] if packed_dt == "f32" else [])
        for center, bias, mode in modes if n != 2111 or cols in (64, 1001, 4096, 16384) else modes[:1]:
            packed = torch.randn(total, device=DEV, generator=gen).to(DT[packed_dt])
            before = packed.clone()
            prev = None if mode == "none" else packed if mode == "in place" else torch.randn(total, device=DEV, generator=gen)
            base = np.zeros(total) if prev is None else _f64(prev)
            whole, dx = guarded(n * cols, DT[dt], DEV)
            scale = float(np.float32(-1.7))
            rs.rs_layer_norm_grad(plan, 1, flat, x, dy, dx, packed, work, bias=bias, eps=1e-3, center=center, prev=prev,
                                  scale=scale, inv_v=mode == "prev")
            assert guard_intact(whole, n * cols)
            sigma = float(np.float32(scale / plan.V)) if mode == "prev" else scale
            grads, sizes = [np.zeros(cols)] * 2, [np.zeros(cols)] * 2
            if n:
                xd, dyd = _f64(x), _f64(dy)
                want, *grads = ON.norm_grad(xd, dyd, w, 1e-3, center)
                h, r, a = _parts(xd, 1e-3, center)
                g = np.abs(dyd * w)
                off = 128 * U * r * (g + g.mean(1, keepdims=True) + (np.abs(h) + a) * (g * (np.abs(h) + a)).mean(1, keepdims=True))
                off += STEP[dt] * (np.abs(want) + off)
                assert (np.abs(_f64(dx).reshape(n, cols) - want) <= off).all(), (n, center, mode)
                sizes = [(np.abs(dyd) * (np.abs(h) + a)).sum(0), np.abs(dyd).sum(0)]
            got = _f64(packed)
            left = np.ones(total, dtype=bool)
            for t, d, size in zip((1, 2) if bias else (1,), grads, sizes):
                at = slice(plan.starts[t], plan.starts[t] + cols)
                left[at] = False
                want = base[at] + sigma * d
                off = (n / 256 + 364) * U * abs(sigma) * size + 2 * U * (np.abs(base[at]) + abs(sigma) * np.abs(d))
                off += STEP[packed_dt] * (np.abs(want) + off)
                assert (np.abs(got[at] - want) <= off).all(), (n, center, mode, t)
            assert np.array_equal(got[left], _f64(before)[left])
    plan.close()


def test_rows_stay_apart(gpu_lib):
    """NaN, infinities and rows of equal values or zeros change their own rows only."""
    import structure_aware_grouped_amd as rs
    plan = _plan(rs, 128)
    gen = torch.Generator(device=DEV).manual_seed(1)
    flat = _gathered(plan, "f32", gen)
    x = torch.randn(8, 128, device=DEV, generator=gen)
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    rs.rs_layer_norm(plan, 1, flat, x, y0, bias=2)
    bad = x.clone()
    bad[1, 5], bad[3, 7], bad[5] = float("nan"), float("inf"), 0.0
    bad[6] = 77.25
    rs.rs_layer_norm(plan, 1, flat, bad, y1, bias=2)
    assert torch.equal(y1[[0, 2, 4, 7]], y0[[0, 2, 4, 7]])
    assert y1[1].isnan().all() and y1[3].isnan().any()
    b = flat[plan.starts[2]:plan.starts[2] + 128]
    assert torch.equal(y1[5], b) and torch.equal(y1[6], b)          # 128 times 77.25 sums exactly
    rs.rs_layer_norm(plan, 1, flat, bad, y1, bias=2, eps=0.0)
    assert y1[5].isnan().all()
    plan.close()


def test_same_bits_again_and_in_a_larger_batch(gpu_lib):
    import structure_aware_grouped_amd as rs
    plan = _plan(rs, 1000)
    gen = torch.Generator(device=DEV).manual_seed(2)
    flat = _gathered(plan, "bf16", gen)
    x = torch.randn(3000, 1000, device=DEV, generator=gen)
    dy = torch.randn(3000, 1000, device=DEV, generator=gen)
    y, z = torch.empty_like(x), torch.empty(17, 1000, device=DEV)
    rs.rs_layer_norm(plan, 1, flat, x, y, bias=2)
    rs.rs_layer_norm(plan, 1, flat, x[:17], z, bias=2)
    assert torch.equal(y[:17], z)
    out = []
    for _ in range(2):
        dx, packed = torch.empty_like(x), torch.zeros(plan.R_mat * plan.S, device=DEV)
        rs.rs_layer_norm_grad(plan, 1, flat, x, dy, dx, packed, rs.rs_layer_norm_workspace(plan, 1, 3000).fill_(255), bias=2)
        out.append((dx, packed))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    plan.close()


def test_other_stream_and_graph(gpu_lib):
    import structure_aware_grouped_amd as rs
    plan = _plan(rs, 512)
    gen = torch.Generator(device=DEV).manual_seed(3)
    flat = _gathered(plan, "bf16", gen)
    x, dy, dx = (torch.zeros(900, 512, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    packed, y = torch.zeros(plan.R_mat * plan.S, device=DEV), torch.zeros_like(x)
    work = rs.rs_layer_norm_workspace(plan, 1, 900)

    def both():
        rs.rs_layer_norm(plan, 1, flat, x, y, bias=2)
        rs.rs_layer_norm_grad(plan, 1, flat, x, dy, dx, packed, work, bias=2, prev=packed)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    for k in range(3):
        x.copy_(torch.randn(900, 512, device=DEV, generator=gen))
        dy.copy_(torch.randn(900, 512, device=DEV, generator=gen))
        start = torch.randn(plan.R_mat * plan.S, device=DEV, generator=gen)
        packed.copy_(start)
        torch.cuda.synchronize()
        if k == 1:
            with torch.cuda.stream(side):
                both()
        else:
            both()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, dx, packed)]
        packed.copy_(start)
        y.zero_(), dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, packed)))
    plan.close()


def test_offsets_past_32_bits(gpu_lib):
    import structure_aware_grouped_amd as rs
    cols, n = 4096, (1 << 20) + 1000           # 2^32 elements and more
    plan = _plan(rs, cols)
    gen = torch.Generator(device=DEV).manual_seed(4)
    flat = _gathered(plan, "bf16", gen)
    x = torch.empty(n, cols, device=DEV, dtype=torch.bfloat16).normal_(generator=gen)
    y = torch.zeros_like(x)
    rs.rs_layer_norm(plan, 1, flat, x, y, bias=2)
    part = torch.empty(1000, cols, device=DEV, dtype=torch.bfloat16)
    for at in (0, n - 1000):
        rs.rs_layer_norm(plan, 1, flat, x[at:at + 1000].clone(), part, bias=2)
        assert torch.equal(part, y[at:at + 1000])
    packed = torch.zeros(plan.R_mat * plan.S, device=DEV)
    dx = torch.zeros_like(x)
    x[1000:n - 1000] = 0
    y[1000:n - 1000] = 0                       # rows without a gradient
    rs.rs_layer_norm_grad(plan, 1, flat, x, y, dx, packed, rs.rs_layer_norm_workspace(plan, 1, n), bias=2)
    xs, ys = (torch.cat([t[:1000], t[n - 1000:]]) for t in (x, y))
    ds, small = torch.zeros_like(xs), torch.zeros_like(packed)
    rs.rs_layer_norm_grad(plan, 1, flat, xs, ys, ds, small, rs.rs_layer_norm_workspace(plan, 1, 2000), bias=2)
    assert torch.equal(ds, torch.cat([dx[:1000], dx[n - 1000:]])) and not dx[1000:n - 1000].any()
    at = slice(plan.starts[1], plan.starts[1] + cols)
    assert torch.allclose(packed[at], small[at], rtol=0, atol=float(600 * U * (ys.abs().float() * 6).sum(0).max()))
    plan.close()


def test_refusals(gpu_lib):
    import structure_aware_grouped_amd as rs
    plan = _plan(rs, 64)
    flat = _gathered(plan, "f32", torch.Generator(device=DEV).manual_seed(5))
    x, y, dx = (torch.zeros(10, 64, device=DEV) for _ in range(3))
    packed, work = torch.zeros(plan.R_mat * plan.S, device=DEV), rs.rs_layer_norm_workspace(plan, 1, 10)
    for kw in ({"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"bias": 1}, {"bias": 0}):
        with pytest.raises(rs.RsError):
            rs.rs_layer_norm(plan, 1, flat, x, y, **kw)
    tile = torch.zeros(1, 1024, device=DEV)
    with pytest.raises(rs.RsError):
        rs.rs_layer_norm(plan, 3, flat, tile, tile.clone())
    for kw in ({"scale": float("inf")}, {"eps": -1e-9}, {"bias": 0}):
        with pytest.raises(rs.RsError):
            rs.rs_layer_norm_grad(plan, 1, flat, x, y, dx, packed, work, **kw)
    with pytest.raises(rs.RsError):
        rs.rs_layer_norm_grad(plan, 1, flat, x, y, dx, packed, work[:-1])
    with pytest.raises(rs.RsError):
        rs.rs_layer_norm_workspace(plan, 1, -1)
    with pytest.raises(rs.RsError):
        rs.rs_layer_norm_workspace(plan, 1, 1 << 31)
    odd = torch.zeros(10 * 64 + 1, device=DEV)[1:].view(10, 64)
    with pytest.raises(rs.RsError):
        rs.rs_layer_norm(plan, 1, flat, odd, y)
    plan.close()
    wide = _plan(rs, 16385)
    with pytest.raises(rs.RsError):
        rs.rs_layer_norm_workspace(wide, 1, 1)
    wide.close()


def test_group_of_a_llama_layer(gpu_lib):
    """The norms of a layer's own plan (bf16 gather, 64 ranks), between its matrices."""
    import structure_aware_grouped_amd as rs
    from workloads import workload
    w = workload(1)
    S, starts, _, _ = rs.rs_plan_build(list(w.specs), w.V)
    plan = rs.rs_plan_load(list(w.specs), w.V, S, starts, w.V, 0)
    at = [s.name for s in w.specs].index("mlp_norm")
    gathered = (torch.randn(w.V * S, device=DEV) * 0.1 + 1).to(torch.bfloat16)
    x = torch.randn(50, 4096, device=DEV).to(torch.bfloat16)
    y = torch.empty_like(x)
    rs.rs_layer_norm(plan, at, gathered, x, y, center=False)
    weight = gathered[starts[at]:starts[at] + 4096].double()
    xd = x.double()
    want = xd / (xd.square().mean(1, keepdim=True) + 1e-5).sqrt() * weight
    assert ((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -16)).all()
    packed = torch.zeros(w.V * S, device=DEV)
    rs.rs_layer_norm_grad(plan, at, gathered, x, x, y, packed, rs.rs_layer_norm_workspace(plan, at, 50), center=False, inv_v=True)
    mine = packed[starts[at]:starts[at] + 4096]
    hat = xd / (xd.square().mean(1, keepdim=True) + 1e-5).sqrt()
    assert ((mine.double() - (xd * hat).sum(0) / w.V).abs() <= 500 * U * (xd * hat).abs().sum(0) / w.V).all()
    packed[starts[at]:starts[at] + 4096] = 0
    assert not packed.any()
    plan.close()
