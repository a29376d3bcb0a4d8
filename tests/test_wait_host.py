"""The bounded wait of the prompt kernels' barriers, on the host: the header's own
loop against a barrier, a stop flag and a clock that a script moves."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# ready at look ``at``, stopped from check ``stop_at`` on; the clock moves ``step`` a reading, and
# with ``done_at_clock`` the phase completes while the clock is read (the waiter stood still there)
PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include "kvq_wait.h"
int main(int argc, char** argv) {
  const long at = atol(argv[1]), stop_at = atol(argv[2]), done_at_clock = atol(argv[3]);
  const unsigned long long step = strtoull(argv[4], 0, 10), limit = strtoull(argv[5], 0, 10);
  long looks = 0, checks = 0, readings = 0;
  bool done = false;
  const bool got = kvq::bounded_wait([&] { return ++looks >= at || done; }, [&] { return ++checks >= stop_at; },
                                     [&] {
                                       if (++readings >= done_at_clock) done = true;
                                       return (uint64_t)(7 + readings * step);
                                     },
                                     limit);
  printf("%d %ld %ld %ld\n", got, looks, checks, readings);
}
"""
NEVER = 1 << 40


@pytest.fixture(scope="module")
def wait(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("wait")
    (at / "wait.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "quantized_kv_cache_02_gb300", "csrc"),
                    str(at / "wait.cpp"), "-o", str(at / "wait")], check=True)

    def run(ready=NEVER, stop=NEVER, clock=NEVER, step=1, limit=1000):
        out = subprocess.run([str(at / "wait"), *(str(x) for x in (ready, stop, clock, step, limit))], check=True,
                             capture_output=True, text=True, timeout=60).stdout
        return [int(x) for x in out.split()]

    return run


def test_ready(wait):
    assert wait(ready=1) == [1, 1, 0, 0]
    assert wait(ready=2) == [1, 2, 0, 0]
    assert wait(ready=500)[:2] == [1, 500]


def test_stop(wait):
    assert wait(stop=1) == [0, 2, 1, 0]
    assert wait(stop=40)[0] == 0


def test_the_limit_ends_it(wait):
    got, looks, checks, readings = wait(step=10, limit=1000)
    assert got == 0 and readings == 102  # the first reading starts the time; 1010 later it is over
    assert looks == 64 * readings + 2    # the last one behind the clock


def test_a_phase_completed_while_the_waiter_stood_still(wait):
    """The reading that passes the limit is also the first after the completion."""
    assert wait(clock=2, step=10 ** 9, limit=10 ** 6)[0] == 1
    assert wait(clock=102, step=10, limit=1000)[0] == 1
