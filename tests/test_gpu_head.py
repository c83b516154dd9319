"""rs_head_loss, rs_head_grad, rs_distill_loss and rs_distill_grad against the
64-bit oracle.

Tolerances, with u = 2^-24 (half an fp32 step). A sum of k products of 16-bit
values in fp32 is off by at most 2 k u of the sum of absolute values (an
addition in the matrix cores by at most two half steps), which bounds the
logits (k = columns), dx (k = rows) and the table's gradient (k = tokens). An
exponential is off by 4 u and by u per unit of its argument, the sum of them by
u per value of its longest chain (64 + 1 + rows / 2048 + 32 values), a logarithm
by 4 u. p - q is then off by p (those of its logit and of the log-sum) and q
(that of a teacher's exponentials), and rounded: for dx to bf16 (2^-8), for the
table's gradient to fp16 (2^-11; its scaled values stay normal down to 2^-29 of
the largest weight) or two fp16 parts (2^-22), and results once more to bf16
where they are."""
import numpy as np
import pytest
import torch

from oracle import head as OH
from tests.gpu_util import guard_intact, guarded
from workloads import TensorSpec

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
SIZES = [(1, 1, 1), (1, 2, 64), (3, 5, 7), (33, 300, 40), (64, 255, 64), (65, 257, 128), (128, 1000, 100), (130, 64, 320),
         (257, 513, 192), (300, 1025, 65), (5, 4099, 264)]


def _plan(rs, rows, cols, V=3, kind=("ROWS", 1, 0)):
    specs = [TensorSpec("before", 37, 5, "ELEM"), TensorSpec("head", rows, cols, *kind),
             TensorSpec("tiles", 32, 32, "TILEMAJOR", 16, 16)]
    S, starts, _, _ = rs.rs_plan_build(specs, V)
    return rs.rs_plan_load(specs, V, S, starts, V, 0)


class Case:
    """Inputs of one call on the device, and what the oracle says of them with its tolerances."""

    def __init__(self, rs, n, rows, cols, top=0, teacher_dt="f32", idx=torch.int64, seed=0, none=0.3, temperature=1.0, scale=1.0):
        rng = np.random.default_rng(seed * 1000 + n + rows + cols)
        self.n, self.rows, self.cols, self.top, self.scale, self.temperature = n, rows, cols, top, scale, temperature
        self.plan = _plan(rs, rows, cols)
        self.at = slice(self.plan.starts[1], self.plan.starts[1] + rows * cols)
        self.total = self.plan.R_mat * self.plan.S
        flat = torch.full((self.total,), float("nan"))
        flat[self.at] = torch.from_numpy(rng.standard_normal(rows * cols)) * (2.0 / np.sqrt(cols))
        self.gathered = flat.to(DEV, torch.bfloat16)
        self.table = self.gathered[self.at].double().cpu().numpy().reshape(rows, cols)
        ids = rng.integers(0, rows, (n, max(top, 1)))
        ids[rng.random(ids.shape) < none / (2 if top else 1)] = rng.choice([-1, -100, rows, rows + 5])
        x = rng.standard_normal((n, cols)) + np.where(rng.random((n, 1)) < 0.5, 1.0, 0.0) * self.table[np.clip(ids[:, 0], 0, rows - 1)]
        self.x = torch.from_numpy(x).to(DEV, torch.bfloat16)
        self.ids = torch.from_numpy(ids if top else ids[:, 0]).to(DEV, idx).contiguous()
        self.teacher = torch.from_numpy(rng.standard_normal((n, top)) * 3).to(DEV, DT[teacher_dt]) if top else None
        if top and n > 3:
            self.teacher[1] = float("-inf")                              # nothing left
            self.teacher[2, : top // 2] = float("-inf")
            self.teacher[3, : top // 2] = torch.finfo(DT[teacher_dt]).min
        w = rng.standard_normal(n) * np.exp(rng.standard_normal(n))
        w[rng.random(n) < 0.1] = 0.0
        self.weights = torch.from_numpy(w).float().to(DEV)

    def host(self):
        f64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        return f64(self.x), self.table, self.ids.cpu().numpy(), f64(self.teacher), f64(self.weights)

    def kw(self):
        return dict(scale=self.scale) if not self.top else dict(scale=self.scale, temperature=self.temperature)

    def targets(self):
        return (self.ids, self.teacher) if self.top else (self.ids,)

    def loss(self, rs, loss, work, **kw):
        f = rs.rs_distill_loss if self.top else rs.rs_head_loss
        f(self.plan, 1, self.gathered, self.x, *self.targets(), loss, work, **self.kw(), **kw)

    def grad(self, rs, loss, dx, packed, work, **kw):
        f = rs.rs_distill_grad if self.top else rs.rs_head_grad
        f(self.plan, 1, self.gathered, self.x, *self.targets(), loss, dx, packed, work, **self.kw(), **kw)

    def work(self, rs, packed=None, piece=0):
        return rs.rs_head_workspace(self.plan, 1, self.n, top=self.top, packed=packed, piece=piece).fill_(255)

    def expect(self, weights=None):
        """loss, dx, dtable and how far each may be off; dx and dtable ahead of their last rounding."""
        x, table, ids, teacher, w = self.host()
        w = np.ones(self.n) if weights is None else w
        loss, p, full, live = OH.losses(x, table, ids, teacher, self.temperature, self.scale)
        dx, dtable, _, _ = OH.gradients(x, table, ids, w, teacher, self.temperature, self.scale)
        c = abs(self.scale) / self.temperature
        l = c * (x @ table.T)
        off_l = 2 * (self.cols + 2) * U * c * (np.abs(x) @ np.abs(table).T) + U * np.abs(l)
        z = np.log(np.exp(l - l.max(1, keepdims=True)).sum(1, keepdims=True)) + l.max(1, keepdims=True)
        off_z = off_l.max(1, keepdims=True) + (110 + self.rows / 2048) * U + 4 * U * np.abs(z) + U * (l.max(1, keepdims=True) - l.min(1, keepdims=True))
        off_p = p * (off_l + off_z + 4 * U + U * np.abs(l - z))
        spread = 0.0 if teacher is None else 40.0 / self.temperature      # of the teacher's logits that count
        off_q = (8 + 2 * spread + self.top) * U if self.top else 0.0
        f = self.temperature ** 2
        gap = np.where(full > 0, np.abs(np.log(np.where(full > 0, full, 1.0))) + np.abs(l - z) + 2, 0.0)
        off_loss = f * (full * (off_l + off_z + (off_q + 8 * U) * gap)).sum(1) + f * 300 * U * (full * gap).sum(1)
        off_d = np.where(live[:, None], off_p + off_q * full + 2 * U * (p + full), 0.0)
        a = np.abs(w * self.temperature * self.scale)[:, None] * live[:, None]
        d = np.abs(p - full) * live[:, None]
        return dict(loss=loss, off_loss=off_loss, dx=dx, dtable=dtable, live=live,
                    off_dx=(a * (off_d + (2.0 ** -8 + 2 * self.rows * U) * (d + off_d))) @ np.abs(table) + 4 * U * np.abs(dx),
                    off_dt={k: (a * (off_d + (step + (2 * self.n + 8) * U) * (d + off_d))).T @ np.abs(x) + a.max(initial=0) * 2.0 ** -38 * np.abs(x).sum(0)
                            for k, step in (("f32", 2.0 ** -22), ("bf16", 2.0 ** -11))})


def _f64(t):
    return t.double().cpu().numpy()


def _check_grad(rs, case, packed_dt, mode="none", weights=True, piece=0, inv_v=False, grad_scale=1.0, want=None):
    want = want or case.expect(case.weights if weights else None)
    n, total = case.n, case.total
    gen = torch.Generator(device=DEV).manual_seed(9)
    packed = torch.randn(total, device=DEV, generator=gen).to(DT[packed_dt])
    before = packed.clone()
    prev = None if mode == "none" else packed if mode == "in place" else torch.randn(total, device=DEV, generator=gen)
    base = 0.0 if prev is None else _f64(prev[case.at]).reshape(case.rows, case.cols)
    whole, dx = guarded(n * case.cols, torch.bfloat16, DEV)
    lwhole, loss = guarded(n, torch.float32, DEV)
    case.grad(rs, loss, dx, packed, case.work(rs, packed, piece), weights=case.weights if weights else None, prev=prev,
              inv_v=inv_v, grad_scale=grad_scale, piece=piece)
    torch.cuda.synchronize()
    assert guard_intact(whole, n * case.cols) and guard_intact(lwhole, n)
    assert (np.abs(_f64(loss) - want["loss"]) <= want["off_loss"]).all()
    off = want["off_dx"] + 2.0 ** -8 * (np.abs(want["dx"]) + want["off_dx"])
    assert (np.abs(_f64(dx).reshape(n, -1) - want["dx"]) <= off).all()
    sigma = float(np.float32(np.float32(grad_scale) / case.plan.V)) if inv_v else float(np.float32(grad_scale))
    result = base + sigma * want["dtable"]
    off = abs(sigma) * want["off_dt"][packed_dt] + 4 * U * (np.abs(base) + abs(sigma) * np.abs(want["dtable"])) * (1 + n // 256)
    off += 2.0 ** -8 * (np.abs(result) + off) if packed_dt == "bf16" else 0.0
    got = _f64(packed)
    assert (np.abs(got[case.at].reshape(case.rows, -1) - result) <= off).all()
    left = np.ones(total, dtype=bool)
    left[case.at] = False
    assert np.array_equal(got[left], _f64(before)[left])


@pytest.mark.parametrize("n,rows,cols", SIZES)
def test_loss(gpu_lib, n, rows, cols):
    import structure_aware_grouped_amd as rs
    for top, idx in ((0, torch.int64), (0, torch.int32), (1, torch.int32), (7, torch.int64), (64, torch.int32)):
        case = Case(rs, n, rows, cols, top=top, idx=idx, teacher_dt="bf16" if top == 7 else "f32", scale=0.75,
                    temperature=2.0 if top == 7 else 0.8 if top == 64 else 1.0)
        want = case.expect()
        whole, loss = guarded(n, torch.float32, DEV)
        case.loss(rs, loss, case.work(rs))
        assert guard_intact(whole, n)
        assert (np.abs(_f64(loss) - want["loss"]) <= want["off_loss"]).all(), (top, idx)
        assert not _f64(loss)[~want["live"]].any()
        case.plan.close()


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("packed_dt", ["f32", "bf16"])
def test_label_gradients(gpu_lib, n, rows, cols, packed_dt):
    import structure_aware_grouped_amd as rs
    case = Case(rs, n, rows, cols, idx=torch.int32 if n % 2 else torch.int64, scale=-1.25)
    _check_grad(rs, case, packed_dt)
    _check_grad(rs, case, packed_dt, mode="prev", weights=False, inv_v=True, grad_scale=-2.0)
    if packed_dt == "f32":
        _check_grad(rs, case, packed_dt, mode="in place", grad_scale=0.5)
    case.plan.close()


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("top,temperature", [(1, 1.0), (5, 2.0), (64, 0.8), (256, 3.0)])
def test_teacher_gradients(gpu_lib, n, rows, cols, top, temperature):
    import structure_aware_grouped_amd as rs
    case = Case(rs, n, rows, cols, top=top, teacher_dt="bf16" if top == 64 else "f32", temperature=temperature, scale=1.5)
    _check_grad(rs, case, "bf16" if top == 5 else "f32", mode="prev" if top == 64 else "none")
    case.plan.close()


@pytest.mark.parametrize("packed_dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,none", [(1100, 0.0), (1100, 0.4), (1100, 0.97), (769, 0.3)])
def test_pieces(gpu_lib, packed_dt, n, none):
    """Several pieces, whole, partly filled and empty ones."""
    import structure_aware_grouped_amd as rs
    case = Case(rs, n, 700, 72, none=none)
    want = case.expect(case.weights)
    for piece in (256, 512, 0):
        for mode in ("none", "prev"):
            _check_grad(rs, case, packed_dt, mode=mode, piece=piece, want=want)
        loss = torch.zeros(n, device=DEV)
        case.loss(rs, loss, case.work(rs, piece=piece), piece=piece)
        assert (np.abs(_f64(loss) - want["loss"]) <= want["off_loss"]).all()
    case.plan.close()


def test_kinds_of_blocks(gpu_lib):
    import structure_aware_grouped_amd as rs
    for kind in (("ELEM", 0, 0), ("TILE", 32, 32), ("FLAT", 512, 0), ("WHOLE", 0, 0)):
        case = Case(rs, 40, 300, 64)
        S, starts, _, _ = rs.rs_plan_build([TensorSpec("head", 300, 64, *kind)], 2)
        plan = rs.rs_plan_load([TensorSpec("head", 300, 64, *kind)], 2, S, starts)
        flat = torch.zeros(2 * S, dtype=torch.bfloat16, device=DEV)
        flat[starts[0]:starts[0] + 300 * 64] = case.gathered[case.at]
        a, b = torch.zeros(40, device=DEV), torch.zeros(40, device=DEV)
        rs.rs_head_loss(plan, 0, flat, case.x, case.ids, a, rs.rs_head_workspace(plan, 0, 40))
        case.loss(rs, b, case.work(rs))
        assert torch.equal(a, b)
        plan.close()
        case.plan.close()


@pytest.mark.parametrize("top", [0, 4])
@pytest.mark.parametrize("packed_dt", ["f32", "bf16"])
def test_no_targets_and_no_tokens(gpu_lib, top, packed_dt):
    import structure_aware_grouped_amd as rs
    for n in (0, 5, 300):
        case = Case(rs, n, 100, 64, top=top)
        case.ids.fill_(-100)
        case.x.fill_(float("nan"))
        for mode in ("none", "prev") + (("in place",) if packed_dt == "f32" else ()):
            packed = torch.full((case.total,), 3.0, device=DEV, dtype=DT[packed_dt])
            prev = None if mode == "none" else packed if mode == "in place" else torch.full((case.total,), -0.0, device=DEV)
            loss, dx = torch.full((n,), 7.0, device=DEV), torch.full((n * 64,), 7.0, device=DEV, dtype=torch.bfloat16)
            case.grad(rs, loss, dx, packed, case.work(rs, packed), prev=prev, grad_scale=-1.0)
            assert not loss.view(torch.int32).any() and not dx.view(torch.int16).any()
            mine = packed[case.at].clone()
            if mode == "in place":
                assert (mine == 3).all()
            else:
                assert not mine.view(torch.int32 if packed_dt == "f32" else torch.int16).any()      # +0.0
            packed[case.at] = 3.0
            assert (packed == 3).all()
        case.plan.close()


def test_what_masked_tokens_hold_does_not_matter(gpu_lib):
    """NaN and infinities in tokens without a target or weight, and in empty places of the teacher."""
    import structure_aware_grouped_amd as rs
    for top in (0, 6):
        case = Case(rs, 200, 300, 96, top=top)
        case.weights[10], case.weights[11] = 0.0, 0.0
        outs = []
        for bad in (False, True):
            live = torch.from_numpy(case.expect()["live"]).to(DEV)
            if bad:
                case.x[~live] = float("nan")
                case.x[10], case.x[11] = float("nan"), float("inf")
                if top:
                    empty = (case.ids < 0) | (case.ids >= 300)
                    case.teacher[empty] = float("nan")
            packed = torch.zeros(case.total, device=DEV)
            loss, dx = torch.zeros(200, device=DEV), torch.zeros(200, 96, device=DEV, dtype=torch.bfloat16)
            case.grad(rs, loss, dx, packed, case.work(rs, packed), weights=case.weights)
            outs.append((loss, dx, packed))
        keep = torch.ones(200, dtype=torch.bool, device=DEV)
        keep[10:12] = False
        assert torch.equal(outs[0][0][keep], outs[1][0][keep])
        assert torch.equal(outs[0][1], outs[1][1]) and torch.equal(outs[0][2], outs[1][2])
        assert bool(live[10]) is False or outs[1][0][10].isnan()
        case.plan.close()


def test_nan_stays_with_its_token(gpu_lib):
    import structure_aware_grouped_amd as rs
    case = Case(rs, 150, 300, 64, none=0.0)
    a, b = torch.zeros(150, device=DEV), torch.zeros(150, device=DEV)
    case.loss(rs, a, case.work(rs))
    case.x[7, 3], case.x[80, 1] = float("nan"), float("inf")
    packed, dx = torch.zeros(case.total, device=DEV), torch.zeros_like(case.x)
    case.grad(rs, b, dx, packed, case.work(rs, packed))
    bad = torch.zeros(150, dtype=torch.bool, device=DEV)
    bad[7] = bad[80] = True
    assert b[bad].isnan().all() and torch.equal(a[~bad], b[~bad])
    assert dx[bad].isnan().all() and not dx[~bad].isnan().any()
    case.plan.close()
    soft = Case(rs, 30, 300, 64, top=5, none=0.0)
    soft.loss(rs, a[:30], soft.work(rs))
    soft.teacher[4, 2], soft.teacher[5, 0] = float("nan"), float("inf")
    soft.loss(rs, b[:30], soft.work(rs))
    assert b[4:6].isnan().all() and torch.equal(a[:4], b[:4]) and torch.equal(a[6:30], b[6:30])
    soft.plan.close()


def test_logits_far_apart(gpu_lib):
    """A softmax of one, underflow of the others, and logits near fp32's largest."""
    import structure_aware_grouped_amd as rs
    case = Case(rs, 64, 300, 64, none=0.0, scale=400.0)
    _check_grad(rs, case, "f32")
    case.plan.close()


def test_the_same_row_many_times(gpu_lib):
    """A teacher that names one row in all its places, in some, and rows at the table's ends."""
    import structure_aware_grouped_amd as rs
    case = Case(rs, 40, 257, 64, top=9, none=0.0)
    case.ids[:10] = 200
    case.ids[10:20, ::2] = 256
    case.ids[20:30, 1:4] = 0
    _check_grad(rs, case, "f32")
    case.plan.close()
    case = Case(rs, 300, 257, 64, none=0.0)
    case.ids.fill_(256)
    _check_grad(rs, case, "bf16")
    case.plan.close()


def test_same_bits_again(gpu_lib):
    import structure_aware_grouped_amd as rs
    case = Case(rs, 500, 3000, 200, top=3)
    outs = []
    for byte in (0, 255):
        packed = torch.zeros(case.total, device=DEV)
        loss, dx = torch.zeros(500, device=DEV), torch.zeros(500, 200, device=DEV, dtype=torch.bfloat16)
        case.grad(rs, loss, dx, packed, case.work(rs, packed).fill_(byte), weights=case.weights)
        alone = torch.zeros(500, device=DEV)
        case.loss(rs, alone, case.work(rs).fill_(byte))
        assert torch.equal(alone, loss)
        outs.append((loss, dx, packed))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    case.plan.close()


@pytest.mark.parametrize("top", [0, 8])
def test_graph_and_streams(gpu_lib, top):
    """Captured once and replayed with other inputs, other numbers of targets among them, between
    eager calls on two streams."""
    import structure_aware_grouped_amd as rs
    case = Case(rs, 600, 900, 128, top=top)
    packed = torch.zeros(case.total, device=DEV)
    loss, dx = torch.zeros(600, device=DEV), torch.zeros(600, 128, device=DEV, dtype=torch.bfloat16)
    works = [case.work(rs, packed, 256) for _ in range(2)]
    call = lambda i: case.grad(rs, loss, dx, packed, works[i], weights=case.weights, prev=packed, piece=256)  # noqa: E731
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(0)
    gen = torch.Generator(device=DEV).manual_seed(0)
    for k, share in enumerate((0.0, 0.5, 1.0, 0.2)):
        case.x.copy_(torch.randn(case.x.shape, device=DEV, generator=gen))
        case.ids.copy_(torch.randint(0, 900, case.ids.shape, device=DEV, generator=gen))
        case.ids[torch.rand(600, device=DEV, generator=gen) < share] = -1
        start = torch.randn(case.total, device=DEV, generator=gen)
        packed.copy_(start)
        torch.cuda.synchronize()
        with torch.cuda.stream(side if k % 2 else torch.cuda.current_stream()):
            call(1)
        torch.cuda.synchronize()
        want = [t.clone() for t in (loss, dx, packed)]
        packed.copy_(start)
        loss.fill_(3), dx.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (loss, dx, packed)))
    case.plan.close()


def test_two_calls_at_once(gpu_lib):
    import structure_aware_grouped_amd as rs
    cases = [Case(rs, 300, 2000, 128, seed=i) for i in range(2)]
    outs = [(torch.zeros(300, device=DEV), torch.zeros(300, 128, device=DEV, dtype=torch.bfloat16), torch.zeros(c.total, device=DEV)) for c in cases]
    for c, o in zip(cases, outs):
        c.grad(rs, *o, c.work(rs, o[2]))
    torch.cuda.synchronize()
    want = [[t.clone() for t in o] for o in outs]
    streams = [torch.cuda.Stream() for _ in cases]
    works = [c.work(rs, o[2]) for c, o in zip(cases, outs)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, o, s, w in zip(cases, outs, streams, works):
            with torch.cuda.stream(s):
                c.grad(rs, *o, w)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))
    for c in cases:
        c.plan.close()


def test_refusals(gpu_lib):
    import structure_aware_grouped_amd as rs
    case = Case(rs, 10, 100, 64)
    packed, loss, dx = torch.zeros(case.total, device=DEV), torch.zeros(10, device=DEV), torch.zeros_like(case.x)
    work = case.work(rs, packed)
    args = (case.plan, 1, case.gathered, case.x, case.ids)
    for kw in ({"scale": float("nan")}, {"piece": 100}, {"piece": -256}, {"piece": 1 << 17}):
        with pytest.raises(rs.RsError):
            rs.rs_head_loss(*args, loss, work, **kw)
    for kw in ({"scale": float("inf")}, {"grad_scale": float("nan")}, {"piece": 255}):
        with pytest.raises(rs.RsError):
            rs.rs_head_grad(*args, loss, dx, packed, work, **kw)
    with pytest.raises(rs.RsError):
        rs.rs_head_loss(*args, loss, case.work(rs)[:-1])
    with pytest.raises(rs.RsError):
        rs.rs_head_grad(*args, loss, dx, packed, work[:-1])
    with pytest.raises(rs.RsError):
        rs.rs_head_loss(case.plan, 2, case.gathered, torch.zeros(10, 32, device=DEV, dtype=torch.bfloat16), case.ids, loss, work)
    for bad in ((10, 257, None, 0), (-1, 0, None, 0), ((1 << 20) + 1, 0, None, 0), (1 << 20, 256 + 1, None, 0), (10, 0, None, 3)):
        with pytest.raises(rs.RsError):
            rs.rs_head_workspace(case.plan, 1, bad[0], top=bad[1], packed=bad[2], piece=bad[3])
    ids, z = torch.zeros(10, 4, device=DEV, dtype=torch.int64), torch.zeros(10, 4, device=DEV)
    big = rs.rs_head_workspace(case.plan, 1, 10, top=4, packed=torch.float32)
    for kw in ({"temperature": 0.0}, {"temperature": -1.0}, {"temperature": float("inf")}, {"temperature": 1e30}, {"scale": float("nan")},
               {"temperature": 1e-30, "scale": 1e30}):
        with pytest.raises(rs.RsError):
            rs.rs_distill_loss(case.plan, 1, case.gathered, case.x, ids, z, loss, big, **kw)
        with pytest.raises(rs.RsError):
            rs.rs_distill_grad(case.plan, 1, case.gathered, case.x, ids, z, loss, dx, packed, big, **kw)
    with pytest.raises(rs.RsError):
        rs.rs_distill_loss(case.plan, 1, case.gathered, case.x, ids[:, :0], z[:, :0], loss, big)
    with pytest.raises(rs.RsError):
        rs.rs_distill_loss(case.plan, 1, case.gathered, case.x, ids, torch.zeros(41, device=DEV)[1:].view(10, 4), loss, big)
    case.plan.close()
