"""Cut tiles of the matrix products pay: a launch whose tiles are cut ends more
than a join costs (24 steps of 256-wide tiles, 30 of smaller ones) ahead of the
same launch with whole tiles, and near the mean where there are tiles for every
workgroup (tests/cpp/matrix_cover.cpp)."""
import random
import re

import pytest

from tests.test_matrix_cover import LAYER, _run, exe  # noqa: F401  (a fixture)

LIST = re.compile(r"\[(\d+) tiles of (\d+), (\d+) cut, \d+ jobs, share ([0-9.]+), behind (-?[0-9.]+), ahead (-?[0-9.]+)\]")


def _lists(exe, shapes, tile=None):  # noqa: F811
    found = [(int(n), int(side), int(cut), float(share), float(behind), float(ahead))
             for n, side, cut, share, behind, ahead in LIST.findall(_run(exe, shapes, tile=tile))]
    assert len(found) == 6
    return found


def _one_matrix(exe, shape, tile=None):  # noqa: F811
    for n, side, cut, share, behind, ahead in _lists(exe, [shape], tile):
        if not cut:
            continue
        # two-part operands (at most 64 rows) count a step three times
        assert ahead > (24 if side == 256 else 30), (shape, side, ahead)
        if n >= (256 if side == 256 else 512):
            assert share <= 1.1 or behind < 25, (shape, side, n, share, behind)


@pytest.mark.parametrize("shape", [(5000, 5000), (5900, 5900), (6001, 5900), (4096, 4096), (8192, 28672), (2880, 2880)])
def test_known_matrices(exe, shape):  # noqa: F811
    _one_matrix(exe, shape)


@pytest.mark.parametrize("seed", range(60))
def test_random_matrices(exe, seed):  # noqa: F811
    rng = random.Random(seed)
    shape = tuple(int(2 ** rng.uniform(7, 13.5)) for _ in range(2))
    _one_matrix(exe, shape, rng.choice([None, None, 64, 128, 256]))


@pytest.mark.parametrize("seed", range(40))
def test_random_groups_do_not_lose_by_their_cuts(exe, seed):  # noqa: F811
    rng = random.Random(seed)
    shapes = [tuple(rng.choice([64, 300, 1000, 1536, 2049, 2880, 4096, 5000, 5900, 6001]) for _ in range(2))
              for _ in range(rng.randint(2, 8))]
    for n, side, cut, share, behind, ahead in _lists(exe, shapes, rng.choice([None, 64, 128, 256])):
        assert not cut or ahead > 0, (shapes, side, ahead)


def test_cuts_of_a_layer(exe):  # noqa: F811
    for n, side, cut, share, behind, ahead in _lists(exe, LAYER):
        assert not cut or ahead > 24
