"""tests/cpp/matrix_lists.cpp from Python: the work lists of the matrix products."""
import os
import re
import shutil
import subprocess
from typing import List, NamedTuple

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "structure_aware_grouped_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
LAYER = [(4096, 4096), (1024, 4096), (1024, 4096), (4096, 4096), (14336, 4096), (14336, 4096), (4096, 14336)]
GRAM, SQUARE, APPLY, SQUARE_PAIRED, GRAM_SINGLE, APPLY_SINGLE = range(6)
_LIST = re.compile(r"\[(\d+) tiles of (\d+), (\d+) cut, (\d+) jobs, share ([0-9.]+), behind (-?[0-9.]+), ahead (-?[0-9.]+)\]")


class Launch(NamedTuple):
    tiles: int
    side: int
    cut: int
    jobs: int
    share: float
    behind: float
    ahead: float


class Lists(NamedTuple):
    launches: List[Launch]
    work: int     # bytes of workspace
    parts: int    # of them the cut tiles' parts


def build(folder) -> str:
    gxx = shutil.which("g++")
    if not gxx or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime_api.h")):
        pytest.skip("needs g++ and the HIP headers")
    out = str(folder / "matrix_lists")
    cmd = [gxx, "-std=c++17", "-O2", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(ROOT, "tests", "cpp", "matrix_lists.cpp"),
           os.path.join(CSRC, "planner.cpp"), "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
           f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}", "-pthread", "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


def lists(exe: str, shapes, parts: int = 1, tile=None, pairs: bool = False, cuts: bool = False) -> Lists:
    """The lists of a plan of these WHOLE tensors; they are checked there to run every step once."""
    env = dict(os.environ, RS_MUON_TILE=str(tile or ""), RS_MUON_PAIRS=str(int(pairs)), RS_MUON_CUTS=str(int(cuts)))
    text = f"{parts} {len(shapes)}\n" + "".join(f"{r} {c}\n" for r, c in shapes)
    r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and "violation" not in r.stdout, r.stdout + r.stderr
    work, cut = (int(v) for v in re.search(r"work (\d+) parts (\d+)", r.stdout).groups())
    found = [Launch(*(int(v) for v in m[:4]), *(float(v) for v in m[4:])) for m in _LIST.findall(r.stdout)]
    assert len(found) == 6
    return Lists(found, work, cut)
