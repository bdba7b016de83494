"""What the producer of the paged attention kernels waits for when it gives up, on the host: the rule
is compiled by the C++ compiler and compared with a bookkeeping of every copy that set out."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = r"""
#include "paged_drain.cuh"
// out: (is V, pair, raw, parity) of every wait; returns how many
extern "C" int drain(int k, int v, uint32_t it, int v_skipped, uint32_t pairs, uint32_t raw_par,
                     uint32_t raw_last, int* out) {
    int n = 0;
    auto put = [&](int is_v, uint32_t pair, bool raw, uint32_t par) {
        out[4 * n] = is_v;
        out[4 * n + 1] = (int)pair;
        out[4 * n + 2] = raw;
        out[4 * n + 3] = (int)par;
        ++n;
    };
    auto on_k = [&](uint32_t pair, uint32_t par) { put(0, pair, false, par); };
    auto on_v = [&](uint32_t pair, bool raw, uint32_t par) { put(1, pair, raw, par); };
    if (k && v) eattn::paged_drain<true, true>(it, v_skipped, pairs, raw_par, raw_last, on_k, on_v);
    else if (k) eattn::paged_drain<true, false>(it, v_skipped, pairs, raw_par, raw_last, on_k, on_v);
    else eattn::paged_drain<false, true>(it, v_skipped, pairs, raw_par, raw_last, on_k, on_v);
    return n;
}
"""


@pytest.fixture(scope="module")
def drain(tmp_path_factory):
    d = tmp_path_factory.mktemp("drain")
    (d / "shim.cpp").write_text(SHIM)
    so = str(d / "shim.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "exact_io_aware_70_b200", "csrc"), str(d / "shim.cpp"), "-o",
                    so], check=True)
    fn = ctypes.CDLL(so).drain

    def call(k, v, it, v_skipped, pairs, raw_par, raw_last):
        out = (ctypes.c_int * (8 * pairs + 8))()
        n = fn(k, v, it, v_skipped, pairs, raw_par, raw_last, out)
        return {tuple(out[4 * i:4 * i + 4]) for i in range(n)}

    return call


@pytest.mark.parametrize("pairs", [2, 3, 4, 5, 6])
@pytest.mark.parametrize("k,v", [(True, True), (True, False), (False, True)])
def test_every_copy_in_flight_is_waited_for(drain, pairs, k, v):
    """A producer that loads K, V or both stops at each place where it can, with every mix of V tiles
    that complete kv_full themselves and ones that are zeroed in between."""
    rng = random.Random(pairs)
    for _ in range(400):
        stop, share = rng.randrange(0, 4 * pairs + 2), rng.choice([0, 0.2, 0.7, 1])
        where = rng.choice((["k"] if k else []) + (["v", "tail"] if v else []) + ["unit"])
        flight = {}                       # slot -> the wait that its last copy's arrival completes
        v_full, v_raw = [0] * pairs, [0] * pairs
        raw_par = raw_last = 0
        it, skipped = 0, False
        while True:
            pair, rnd = it % pairs, it // pairs
            if it == stop and where == "unit":
                break
            if k:
                if it == stop and where == "k" and rnd > 0:
                    break
                flight[("k", pair)] = (0, pair, 0, rnd & 1)
            if v:
                raw = rng.random() < share
                if it == stop and where == "v" and rnd > 0:     # the slot is another tile's still
                    it, skipped = it + 1, True
                    break
                if it == stop and where == "tail" and raw:
                    flight.pop(("v", pair), None)               # its last copy has been used up
                    it, skipped = it + 1, True
                    break
                if raw:
                    flight[("v", pair)] = (1, pair, 1, v_raw[pair] & 1)
                    v_raw[pair] += 1
                    raw_par, raw_last = raw_par ^ (1 << pair), raw_last | (1 << pair)
                else:
                    flight[("v", pair)] = (1, pair, 0, v_full[pair] & 1)
                    raw_last &= ~(1 << pair)
                v_full[pair] += 1         # (a zeroed tile completes kv_full in the end, too)
            it += 1
            if it > stop:                 # the place cannot be reached at that tile
                break
        waits = drain(k, v, it, skipped, pairs, raw_par, raw_last)
        assert set(flight.values()) <= waits, (where, stop, it)
        # and for nothing that has not set out: such a wait would run into its limit
        for is_v, pair, raw, par in waits:
            last = (v_raw if raw else v_full)[pair] - 1 if is_v else (it - 1 - pair) // pairs
            assert last >= 0 and par == last & 1, (where, stop, it)
