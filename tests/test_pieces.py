"""The routed calls' pieces of rows (csrc/pieces.hpp) read and write nothing outside
their arrays: the header compiled for the host with stand-ins for the device
builtins, under AddressSanitizer (tests/sanitize/pieces_driver.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = os.environ.get("AMDCLANGXX", "/opt/rocm/bin/amdclang++")

HOST_DEVICE_HPP = """#pragma once
#include <stdint.h>
#define __device__
#define __forceinline__ inline
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
inline unsigned host_alignbyte(unsigned hi, unsigned lo, unsigned s) {
  return (unsigned)((((uint64_t)hi << 32) | lo) >> (8 * (s & 3)));
}
#define __builtin_amdgcn_alignbyte host_alignbyte
template <typename T>
unsigned pack2(float a, float b);
"""


@pytest.mark.skipif(not os.path.exists(CLANG), reason="no clang++ with _Float16")
def test_pieces_stay_inside_their_arrays(tmp_path):
    for f in ("dequant_gemv_amd/csrc/pieces.hpp", "tests/sanitize/pieces_driver.cpp"):
        shutil.copy(os.path.join(ROOT, f), tmp_path)
    (tmp_path / "device.hpp").write_text(HOST_DEVICE_HPP)
    (tmp_path / "rows.hpp").write_text("#pragma once\n")
    exe = str(tmp_path / "pieces_driver")
    r = subprocess.run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address", "-fno-sanitize-recover=all",
                        str(tmp_path / "pieces_driver.cpp"), "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "pieces: ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
