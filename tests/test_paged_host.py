"""Host-side choices and checks of the serving entry points (no GPU needed)."""
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


@pytest.mark.parametrize("what", ["page_size", "num_pages", "negative", "rows", "free", "keep_first",
                                  "keep_last", "select_page_size", "num_sel", "max_pages"])
def test_sizes_beyond_32_bits_are_refused(what, monkeypatch):
    """The C calls take sizes as 32-bit ints: 2^32 + 16 must not pass as 16."""
    import torch

    import exact_io_aware_70_b200 as ea

    big = 2 ** 32 + 16
    monkeypatch.setattr(ea, "_pointers", lambda what, names, dtypes, ts: (0, [0x10000] * len(ts)))
    monkeypatch.setattr(ea, "_rows", lambda t, name, dev: (0x10000, t.shape[1] * t.shape[2]))
    launched = []
    monkeypatch.setattr(ea, "_launch", lambda fn, name, dev, args, stream: launched.append(args))

    def i32(*shape):
        return torch.zeros((1,) * len(shape), dtype=torch.int32).expand(*shape)

    def tables(page_size=16, num_pages=50, rows=4, free=50):
        ea.attn_page_tables(i32(2), i32(2), i32(free), i32(1), i32(1), i32(2, 8), i32(2), i32(3),
                            i32(rows), page_size, num_pages)

    def select(keep_first=0, keep_last=1, page_size=16, num_sel=4, max_pages=8):
        q, kb = torch.zeros((4, 2, 64)), torch.zeros((50, 1, 2, 64))
        ea.attn_page_select(q, kb, i32(2, max_pages), i32(3), i32(2), i32(4, 1, num_sel), page_size,
                            keep_first, keep_last, i32(256))

    tables()
    select()
    assert len(launched) == 2                    # these pass
    with pytest.raises(ValueError, match="32 bits"):
        {"page_size": lambda: tables(page_size=big), "num_pages": lambda: tables(num_pages=big),
         "negative": lambda: tables(page_size=16 - 2 ** 32), "rows": lambda: tables(rows=big),
         "free": lambda: tables(free=big), "keep_first": lambda: select(keep_first=big - 16),
         "keep_last": lambda: select(keep_last=1 - 2 ** 32),
         "select_page_size": lambda: select(page_size=big), "num_sel": lambda: select(num_sel=big),
         "max_pages": lambda: select(max_pages=big)}[what]()
    assert len(launched) == 2
    with pytest.raises(ValueError, match="32 bits"):
        ea.attn_page_select_workspace_bytes(4, 2, big)


def test_smoke_runs_the_serving_step_without_the_test_modules():
    """The step of smoke() needs helper modules alone, not the tests (nor pytest)."""
    import ast
    tree = ast.parse(open(os.path.join(ROOT, "__graft_entry__.py")).read())
    fn = next(f for f in tree.body if getattr(f, "name", "") == "_smoke_serving")
    names = {a.name for n in ast.walk(fn) if isinstance(n, (ast.Import, ast.ImportFrom))
             for a in n.names}
    assert names == {"torch", "exact_io_aware_70_b200", "paged_util"}
    assert "test_gpu_serving" not in ast.unparse(tree)
