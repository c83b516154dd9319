"""The sizes that the embedding calls accept and refuse, without a GPU
(tests/cpp/embed_limits.cpp): columns are numbered in 32 bits by the lookup,
and every launch stays under 2^32 work-items."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "structure_aware_grouped_amd")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
OK, ERANGE = 0, -7


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime_api.h")):
        pytest.skip("needs g++ and the HIP headers")
    out = str(tmp_path_factory.mktemp("limits") / "embed_limits")
    cmd = [gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(LIB, "csrc"),
           os.path.join(ROOT, "tests", "cpp", "embed_limits.cpp"), os.path.join(LIB, "librs_hip.so"),
           f"-Wl,-rpath,{LIB}", "-L", os.path.join(ROCM, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}",
           "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(rows, cols, n_ids):
        r = subprocess.run([out], input=f"{rows} {cols} {n_ids}\n", capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        return tuple(int(v) for v in r.stdout.split())

    return ask


@pytest.mark.parametrize("rows,cols,n_ids", [
    (1, 1, 0), (1, 1, 2 ** 26 - 1), (2 ** 27 - 8, 1, 2 ** 26 - 1), (2 ** 27 - 8, 128, 64), (1, 2 ** 31 - 1, 4),
    (8, 2 ** 31 - 8, 4), (2 ** 24, 1024, 2 ** 23), (131072, 8192, 65536)])
def test_accepted(ask, rows, cols, n_ids):
    status, size = ask(rows, cols, n_ids)
    assert status == OK and size >= n_ids * 8


@pytest.mark.parametrize("rows,cols,n_ids", [
    # a row's units would not fit 32 bits: 2^32 + 1 columns would count as one, and offsets in a
    # row would wrap from 2^32 columns on
    (1, 2 ** 32 + 1, 1), (2, 2 ** 32 + 64, 1), (1, 2 ** 33, 1), (1, 2 ** 33 - 1, 1), (3, 2 ** 32, 0), (4, 2 ** 31, 1),
    # 2^24 workgroups of 256 in the pass over the whole table
    (2 ** 27 - 1, 1, 2 ** 26 - 1), (2 ** 27 - 7, 1, 1), (2 ** 27, 1, 1),
    (2 ** 24 + 1, 1024, 1), (100, 1, 2 ** 26), (100, 2 ** 20, 2 ** 13 + 1)])
def test_refused(ask, rows, cols, n_ids):
    assert ask(rows, cols, n_ids) == (ERANGE, -1)
