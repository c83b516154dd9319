"""Two-part operands for every matrix (rs_plan_load_with's muon_parts): the
options that are refused, and the work lists and workspace that they give
(tests/cpp/matrix_lists.cpp)."""
import ctypes
import random

import pytest

from tests.matrix_lists import LAYER, build, lists
from workloads import TensorSpec


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    return build(tmp_path_factory.mktemp("lists"))


def _load(rs, specs, options):
    from structure_aware_grouped_amd import binding as b
    S, starts, _, _ = rs.rs_plan_build(specs, 1)
    h = ctypes.c_void_p(7)
    status = b.load().rs_plan_load_with(b.specs_array(specs), 1, 1, S, b._i64(starts), 1, 0, options, ctypes.byref(h))
    return status, h.value


@pytest.mark.parametrize("parts", [-1, 3, 1 << 30])
def test_other_numbers_of_parts_are_refused(parts):
    import structure_aware_grouped_amd as rs
    from structure_aware_grouped_amd import binding as b
    specs = [TensorSpec("w", 128, 128, "WHOLE")]
    assert _load(rs, specs, ctypes.byref(b.PlanOptionsC(muon_parts=parts))) == (b.RS_EINVAL, None)
    assert "muon_parts" in b.load().rs_last_error().decode()


def test_reserved_options_are_refused():
    import structure_aware_grouped_amd as rs
    from structure_aware_grouped_amd import binding as b
    for k in range(7):
        options = b.PlanOptionsC()
        options.reserved[k] = 1
        assert _load(rs, [TensorSpec("w", 128, 128, "WHOLE")], ctypes.byref(options)) == (b.RS_EINVAL, None)


@pytest.mark.parametrize("tile", [None, 64, 128, 256])
@pytest.mark.parametrize("shapes", [[(65, 65)], [(1024, 4096)], [(128, 2880), (333, 1001), (40, 900)], LAYER,
                                    [(5760, 2880), (2880, 2880)] * 8])
def test_every_step_once_with_two_parts(exe, shapes, tile):
    lists(exe, shapes, 2, tile, pairs=True)       # two-part matrices have no paired steps, asked for or not


def _stated(rows, cols, parts, pad=64):
    """The workspace that rs.h states for one matrix, with its sides padded to `pad`."""
    m, n = (-(-v // pad) * pad for v in (min(rows, cols), max(rows, cols)))
    if min(rows, cols) < 2 or (min(rows, cols) <= 64 and max(rows, cols) <= 256):
        return 0
    if parts == 2 or min(rows, cols) <= 64:
        return 12 * m * n + 8 * m * m
    paired = min(rows, cols) >= 1024 and 2 * max(rows, cols) >= 3 * min(rows, cols)
    return 8 * m * n + (8 if paired else 4) * m * m


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("seed", range(25))
def test_workspace_is_as_stated(exe, seed, parts):
    rng = random.Random(seed)
    shapes = [(rng.choice([2, 17, 64, 65, 300, 1000, 1024, 1100, 2049, 5000, 8192]), rng.choice([2, 33, 64, 129, 300, 777, 2880, 6000, 20000]))
              for _ in range(rng.randint(1, 6))] if seed else [(2880, 5760)] * 16
    found = lists(exe, shapes, parts)
    work, cut = found.work, found.parts
    stated, bare = (sum(_stated(*s, parts, pad) for s in shapes) for pad in (64, 1))
    assert cut <= 128 << 20
    assert bare <= work - cut <= 1.01 * stated + 8192 * len(shapes), (shapes, work, cut, stated)
