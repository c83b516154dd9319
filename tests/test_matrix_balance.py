"""Cut tiles of the matrix products pay: a launch whose tiles are cut ends more
than a join costs (24 steps of 256-wide tiles, 30 of smaller ones) ahead of the
same launch with whole tiles, and near the mean where there are tiles for every
workgroup (tests/cpp/matrix_lists.cpp)."""
import random

import pytest

from tests.matrix_lists import LAYER, build, lists


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    return build(tmp_path_factory.mktemp("lists"))


def _one_matrix(exe, shape, tile=None):
    for x in lists(exe, [shape], tile=tile).launches:
        if not x.cut:
            continue
        assert x.ahead > (24 if x.side == 256 else 30), (shape, x)
        if x.tiles >= (256 if x.side == 256 else 512):
            assert x.share <= 1.1 or x.behind < 25, (shape, x)


@pytest.mark.parametrize("shape", [(5000, 5000), (5900, 5900), (6001, 5900), (4096, 4096), (8192, 28672), (2880, 2880)])
def test_known_matrices(exe, shape):
    _one_matrix(exe, shape)


@pytest.mark.parametrize("seed", range(60))
def test_random_matrices(exe, seed):
    rng = random.Random(seed)
    shape = tuple(int(2 ** rng.uniform(7, 13.5)) for _ in range(2))
    _one_matrix(exe, shape, rng.choice([None, None, 64, 128, 256]))


@pytest.mark.parametrize("seed", range(40))
def test_random_groups_do_not_lose_by_their_cuts(exe, seed):
    rng = random.Random(seed)
    shapes = [tuple(rng.choice([64, 300, 1000, 1536, 2049, 2880, 4096, 5000, 5900, 6001]) for _ in range(2))
              for _ in range(rng.randint(2, 8))]
    for x in lists(exe, shapes, tile=rng.choice([None, 64, 128, 256])).launches:
        assert not x.cut or x.ahead > 0, (shapes, x)


def test_cuts_of_a_layer(exe):
    for x in lists(exe, LAYER).launches:
        assert not x.cut or x.ahead > 24
