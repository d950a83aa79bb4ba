"""Sizes of the routed calls against what a launch takes (fewer than 2^32 work items a
dimension): the C entry points refuse what no launch can take and accept what
include/qroute.h promises, with the launchers' own grid arithmetic behind stubs
(tests/sanitize/route_grid_driver.cpp, host code only)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "dequant_gemv_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
A = 0x7F0000000000  # an aligned fake device address, never dereferenced
G = 1 << 40         # far enough apart for any size used here


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_no_accepted_call_has_too_large_a_grid(tmp_path):
    exe = str(tmp_path / "route_grid_driver")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-x", "hip", "--cuda-host-only", "-O1", "-g", "-std=c++17",
                        "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "abi.hip"),
                        os.path.join(CSRC, "abi_route.hip"), os.path.join(SAN, "launch_stubs.cpp"),
                        os.path.join(SAN, "route_grid_driver.cpp"), "-o", exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "route grids: ok" in r.stdout, (r.stdout + r.stderr)[-3000:]


def test_sizes_past_a_launch_are_refused_by_the_library():
    from dequant_gemv_amd import qgemv as q

    lib = q.lib()
    p = [A + i * G for i in range(6)]
    t, c = 1 << 24, 2056  # 257 pieces a row: more than 2^32 in all
    assert lib.qroute_gather(p[0], p[1], None, p[2], 1, t, 1, c, None) == q.QGEMV_E_SHAPE
    assert lib.qroute_combine(p[0], 1, p[1], None, p[2], 1, t, 1, c, None) == q.QGEMV_E_SHAPE
    assert lib.qroute_combine_grad(p[0], 1, p[1], 1, p[2], p[3], p[4], p[5], t, 1, c, None) == q.QGEMV_E_SHAPE
    # one slot a weight set, 2^24 workgroups of 256 threads
    assert lib.qgemm_tq1_routed(p[0], p[1], None, p[2], p[3], 0, 1024, 1, 1024, 1 << 20, 256, None) == q.QGEMV_E_SHAPE
