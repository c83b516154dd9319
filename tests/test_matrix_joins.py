"""That tiles are cut where tests of the joins count on it: every product list
under RS_MUON_CUTS=1, and the last product of larger matrices by the plan's own
choice (tests/cpp/matrix_cover.cpp, which also finds every step once)."""
import re

import pytest

from tests.test_gpu_muon import SHAPES
from tests.test_gpu_muon_joins import LARGE
from tests.test_matrix_cover import _run, exe  # noqa: F401  (a fixture)

GRAM, SQUARE, APPLY, SQUARE_PAIRED, GRAM_SINGLE, APPLY_SINGLE = range(6)


def _cuts(exe, shapes, tile=None):  # noqa: F811
    out = _run(exe, shapes, tile=tile)
    assert out.startswith("ok"), out
    return [(int(n), int(cut)) for n, cut in re.findall(r"\[(\d+) tiles of \d+, (\d+) cut", out)]


@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("pairs", ["0", "1"])
def test_forced_cuts_reach_every_product(exe, tile, pairs, monkeypatch):  # noqa: F811
    monkeypatch.setenv("RS_MUON_CUTS", "1")
    monkeypatch.setenv("RS_MUON_PAIRS", pairs)
    cuts = _cuts(exe, SHAPES, tile)
    for w in (GRAM, SQUARE, APPLY) + ((SQUARE_PAIRED,) if pairs == "1" else ()):
        assert cuts[w][1] >= cuts[w][0] // 2, (w, cuts[w])


@pytest.mark.parametrize("shape", LARGE)
def test_the_last_product_of_larger_matrices_is_cut(exe, shape):  # noqa: F811
    cuts = _cuts(exe, [shape])
    assert all(cuts[w][1] > 0 for w in (GRAM, SQUARE, APPLY)), cuts
