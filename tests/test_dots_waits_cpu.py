"""The wait counts of the staged dots (csrc/mhc_waits.h) against the order in which a wave
asks for its loads: what a unit reads has landed, whatever is left in flight."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mhc_hyper_connection_token_amd", "csrc")
UNIT = 5  # loads of a unit, any number


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("waits")
    src, so = d / "waits.cpp", d / "waits.so"
    src.write_text('#include "mhc_waits.h"\n'
                   'extern "C" int in_flight(int s, int c, int n)'
                   '{ return mhc::dots_in_flight(s, c, n); }\n'
                   'extern "C" int dy_loads() { return mhc::kDyLoads; }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", so, src], check=True)
    return ctypes.CDLL(str(so))


def _stale(in_flight, dy_loads, S, slices):
    """(unit, what) of every read of something that may still be in flight."""
    asked, found = [], []

    def ask(what, n):
        asked.extend([what] * n)

    ask(("dy", 0), dy_loads)
    ask(("unit", 0), UNIT)
    ask(("unit", 1), UNIT)
    for u in range(S * slices):
        sl, c = divmod(u, S)
        late = asked[len(asked) - in_flight(S, c, u):]
        reads = [("unit", u)] + ([("dy", sl)] if c == 0 else [])
        found += [(u, r) for r in reads if r in late]
        if c == 0:
            ask(("dy", sl + 1), dy_loads)
        ask(("unit", u + 2), UNIT)
    return found


@pytest.mark.parametrize("S", range(1, 9))
def test_what_a_unit_reads_has_landed(waits, S):
    def count(s, c, u):
        return waits.in_flight(s, c, UNIT)
    assert _stale(count, waits.dy_loads(), S, 6) == []
    # and no wait is for more than that: one load more in flight would be too many
    assert _stale(lambda s, c, u: count(s, c, u) + 1, waits.dy_loads(), S, 6)


def test_a_count_that_leaves_dy_in_flight_is_found():
    """With one stream every unit begins a slice: leaving the four loads of dy in flight
    after each of them is a read of dy that may not have landed; with more it is not."""
    def loose(s, c, u):
        return UNIT + (4 if c == 1 % s and u > 0 else 0)
    assert _stale(loose, 4, 1, 6)[0] == (1, ("dy", 1))
    assert all(_stale(loose, 4, S, 6) == [] for S in range(2, 9))
