"""The clock of the kernels' bounded waits (csrc/wait_clock.cuh), compiled for the
host: a wait that goes on ends after two seconds, and time in which the context
did not run does not end one."""
import ctypes
import os
import shutil
import subprocess

import pytest

from unpermute_stable_counting_gb300 import _build

SOURCE = """
#include "wait_clock.cuh"
extern "C" long readings(const unsigned long long* ns, long n) {  // until the limit; -1: not reached
    mr::WaitClock c;
    for (long i = 0; i < n; ++i)
        if (c.out(ns[i])) return i + 1;
    return -1;
}
"""


@pytest.fixture(scope="module")
def readings(tmp_path_factory):
    cxx = shutil.which("g++") or pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("wait_clock")
    (at / "clock.cpp").write_text(SOURCE)
    lib = str(at / "clock.so")
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", _build.CSRC, str(at / "clock.cpp"), "-o", lib],
                   check=True)
    f = ctypes.CDLL(lib).readings
    f.restype = ctypes.c_long
    return lambda ns: f((ctypes.c_uint64 * len(ns))(*ns), len(ns))


S = 1_000_000_000


@pytest.mark.parametrize("start", [0, 123456789, (1 << 42) - 1_500_000_000, 1 << 62])
@pytest.mark.parametrize("step", [2_000, 100_000, 3_000_000, 90_000_000])
def test_a_wait_ends_after_two_seconds(readings, start, step):
    n = readings([start + i * step for i in range(4 * S // step)])
    assert 2 * S * 0.99 <= (n - 1) * step <= 2 * S * 1.05 + step


def test_time_that_did_not_pass_for_the_kernel_does_not_end_a_wait(readings):
    """Suspended for 3 s, then for an hour, between readings 10 us apart."""
    ns = [i * 10_000 for i in range(100)]
    for pause in (3 * S, 3600 * S):
        ns += [ns[-1] + pause + i * 10_000 for i in range(100)]
    assert readings(ns) == -1


def test_readings_far_apart_end_a_wait_too(readings):
    """However slow the polls are, a bounded number of them ends it."""
    assert readings([i * 5 * S for i in range(100)]) == 21
