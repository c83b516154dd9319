"""The work lists of the matrix products, checked on the host step by step
(tests/cpp/matrix_cover.cpp, which includes plan.cpp). Planted mistakes are
reported."""
import os
import random
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "structure_aware_grouped_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
LAYER = [(4096, 4096), (1024, 4096), (1024, 4096), (4096, 4096), (14336, 4096), (14336, 4096), (4096, 14336)]


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime_api.h")):
        pytest.skip("needs g++ and the HIP headers")
    out = str(tmp_path_factory.mktemp("cover") / "matrix_cover")
    cmd = [gxx, "-std=c++17", "-O2", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(ROOT, "tests", "cpp", "matrix_cover.cpp"),
           os.path.join(CSRC, "planner.cpp"), "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
           f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}", "-pthread", "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


def _run(exe, shapes, plant=0, tile=None):
    env = dict(os.environ)
    env.pop("RS_MUON_TILE", None)
    if tile:
        env["RS_MUON_TILE"] = str(tile)
    text = f"{len(shapes)}\n" + "".join(f"{r} {c}\n" for r, c in shapes)
    r = subprocess.run([exe] + ([str(plant)] if plant else []), input=text, capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0, r.stderr
    return r.stdout.strip()


@pytest.mark.parametrize("tile", [None, 64, 128, 256])
@pytest.mark.parametrize("shapes", [[(64, 48)], [(2, 2)], [(2, 100000)], [(1024, 4096)], [(128, 2880), (333, 1001)],
                                    [(4096, 4096)], [(8192, 28672)], LAYER, [(5760, 2880), (2880, 2880)] * 8,
                                    [(16, 16)] * 700])
def test_every_step_once(exe, shapes, tile):
    out = _run(exe, shapes, tile=tile)
    assert out.startswith("ok"), out


@pytest.mark.parametrize("seed", range(30))
def test_random_groups(exe, seed):
    rng = random.Random(seed)
    shapes = [(rng.choice([2, 17, 64, 65, 300, 1000, 2049, 5000]), rng.choice([2, 33, 64, 129, 777, 2880, 6000]))
              for _ in range(rng.randint(1, 12))]
    out = _run(exe, shapes, tile=rng.choice([None, 64, 128, 256]))
    assert out.startswith("ok"), out


def test_large_products_are_shared_evenly(exe):
    """With at least as many tiles as workgroups the last one ends at most a tenth behind the mean,
    or less than 25 steps: cut tiles need a second launch, so they are cut only where that saves more
    than 24 steps (kMatJoinSteps) over the mean, which is rounded up to whole steps. So 700 tiles of
    64 steps on 256 workgroups, which end after 3 * 64 = 192 steps, 17 behind the mean, stay whole."""
    for shapes in (LAYER, [(8192, 28672)], [(5760, 2880), (2880, 2880)] * 8):
        found = re.findall(r"share ([0-9.]+), behind ([0-9.]+)", _run(exe, shapes, tile=256))
        assert found
        for share, behind in found:
            assert float(share) <= 1.1 or float(behind) < 25, (shapes, share, behind)


@pytest.mark.parametrize("plant", [1, 2, 3, 4])
def test_planted_mistakes_are_reported(exe, plant):
    assert _run(exe, LAYER, plant=plant).startswith("violation")
