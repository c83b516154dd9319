"""The sizes that the head's and layer norm's calls accept and refuse, without a
GPU (tests/cpp/head_limits.cpp), and that a workspace never gets smaller for
more tokens, for gradients or for a teacher."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "structure_aware_grouped_amd")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
OK, EINVAL, EDTYPE, ERANGE = 0, -1, -4, -7
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime_api.h")):
        pytest.skip("needs g++ and the HIP headers")
    out = str(tmp_path_factory.mktemp("limits") / "head_limits")
    cmd = [gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(LIB, "csrc"),
           os.path.join(ROOT, "tests", "cpp", "head_limits.cpp"), os.path.join(LIB, "librs_hip.so"),
           f"-Wl,-rpath,{LIB}", "-L", os.path.join(ROCM, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}",
           "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(rows, cols, n, top=0, grad=0, dt=F32, piece=0):
        r = subprocess.run([out], input=f"{rows} {cols} {n} {top} {grad} {dt} {piece}\n", capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        v = [int(x) for x in r.stdout.split()]
        return v[:2], v[2:]

    return ask


@pytest.mark.parametrize("rows,cols,n,top,piece", [
    (1, 1, 0, 0, 0), (1, 1, 1, 1, 256), (2 ** 21, 2 ** 12, 2 ** 20, 256, 0), (2 ** 17, 2 ** 16, 2 ** 17, 0, 65536),
    (131072, 4096, 16384, 0, 0), (2 ** 21 - 1, 4095, 2 ** 20, 255, 512), (2, 2 ** 16, 1, 0, 0)])
def test_accepted(ask, rows, cols, n, top, piece):
    for grad in (0, 1):
        for dt in (F32, BF16):
            (status, size), _ = ask(rows, cols, n, top, grad, dt, piece)
            assert status == OK and size >= 2 * n * cols


@pytest.mark.parametrize("rows,cols,n,top", [
    (2 ** 21 + 1, 1, 1, 0), (1, 2 ** 16 + 1, 1, 0), (1, 1, 2 ** 20 + 1, 0), (2 ** 18, 2 ** 16, 1, 0), (2 ** 21, 4097, 1, 0),
    (1, 2 ** 16, 2 ** 17 + 1, 0), (2 ** 40, 2 ** 20, 1, 0), (2 ** 31, 1, 1, 0), (1, 1, 2 ** 62, 0), (1, 1, 2 ** 62, 256)])
def test_refused(ask, rows, cols, n, top):
    for grad in (0, 1):
        assert ask(rows, cols, n, top, grad)[0] == [ERANGE, -1]


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n=1, top=-1), dict(n=1, top=257), dict(n=1, piece=-256), dict(n=1, piece=255),
                                dict(n=1, piece=65792), dict(n=1, grad=2), dict(n=1, dt=7)])
def test_bad_arguments(ask, kw):
    status, size = ask(100, 64, **kw)[0]
    assert status in (EINVAL, EDTYPE, ERANGE) and size == -1


@pytest.mark.parametrize("rows,cols", [(1, 1), (300, 40), (4099, 264), (131072, 4096), (9, 4096)])
def test_one_workspace_serves_less(ask, rows, cols):
    last = 0
    for n in (0, 1, 64, 65, 128, 129, 256, 257, 1000, 4096, 8192, 8193, 16384):
        sizes = [ask(rows, cols, n, grad=g)[0][1] for g in (0, 1)]
        taught = [ask(rows, cols, n, top=33, grad=g)[0][1] for g in (0, 1)]
        assert sizes[0] <= sizes[1] <= taught[1] and sizes[0] <= taught[0] <= taught[1]
        assert sizes[0] >= last
        last = sizes[0]


@pytest.mark.parametrize("cols,n,status", [(16384, 2 ** 31 - 1, OK), (1, 0, OK), (16385, 1, ERANGE), (8, 2 ** 31, ERANGE),
                                           (2 ** 40, 1, ERANGE), (8, -1, EINVAL)])
def test_layer_norm(ask, cols, n, status):
    got, size = ask(1, cols, n)[1]
    assert got == status and (size >= 0) == (status == OK)
