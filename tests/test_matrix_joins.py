"""That tiles are cut where tests of the joins count on it: every product list
under RS_MUON_CUTS=1, and the last product of larger matrices by the plan's own
choice (tests/cpp/matrix_lists.cpp, which also finds every step once)."""
import pytest

from tests.matrix_lists import APPLY, GRAM, SQUARE, SQUARE_PAIRED, build, lists
from tests.test_gpu_muon import SHAPES
from tests.test_gpu_muon_joins import LARGE


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    return build(tmp_path_factory.mktemp("lists"))


@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("parts,pairs", [(1, False), (1, True), (2, False)])
def test_forced_cuts_reach_every_product(exe, tile, parts, pairs):
    found = lists(exe, SHAPES, parts, tile, pairs, cuts=True).launches
    for w in (GRAM, SQUARE, APPLY) + ((SQUARE_PAIRED,) if pairs else ()):
        assert found[w].cut >= found[w].tiles // 2, (w, found[w])


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("shape", LARGE)
def test_the_last_product_of_larger_matrices_is_cut(exe, shape, parts):
    found = lists(exe, [shape], parts).launches
    assert all(found[w].cut > 0 for w in (GRAM, SQUARE, APPLY)), found
