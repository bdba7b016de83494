"""Host-side choices of the serving entry points, compiled without CUDA."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = r"""
#include "paged_host.cuh"
extern "C" int ctas(long long rows, int threads, int fit) {
    return eattn::tables_ctas(rows, threads, fit != 0);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("host")
    (d / "shim.cpp").write_text(SHIM)
    so = str(d / "shim.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "exact_io_aware_70_b200", "csrc"), str(d / "shim.cpp"), "-o",
                    so], check=True)
    lib = ctypes.CDLL(so)
    lib.ctas.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return lib


@pytest.mark.parametrize("rows", [1, 1024, 1025, 2048, 2049, 8192, 8193, 47000, 2 ** 30])
def test_block_tables_take_no_cluster_that_does_not_fit(lib, rows):
    narrow, wide = lib.ctas(rows, 1024, 0), lib.ctas(rows, 1024, 1)
    assert narrow in (1, 2, 8) and narrow == min(wide, 8)
    assert wide == (1 if rows <= 1024 else 2 if rows <= 2048 else 8 if rows <= 8192 else 16)
